// gs_gated_ff_fwd and gs_gated_ff_bwd: the gated feed-forward block.
//
//   g = x Wg^T, u = x Wu^T, h = act(g) u, y = h Wd^T
// and back
//   gh = gy Wd, gg = gh u act'(g), gu = gh act(g),
//   gx = gg Wg + gu Wu, gWg = gg^T x, gWu = gu^T x, gWd = gy^T h
//
// Six products of 2 rows channels hidden operations for every three of the
// forward pass's, on the matrix unit; what stands between them is done on the
// accumulators: a tile holds the same columns of both projections, so h leaves
// the first kernel finished, and gg and gu leave the backward's first.
//
// Roundings: sums are fp32. h, gg and gu are rounded to the inputs' type, in
// which the matrix unit takes them. g and u are kept for the backward pass in
// fp32: in 16 bits their roundings would add to those of gg and gu.
#include "product.h"

namespace gs {

enum { ACT_SILU = 0, ACT_GELU = 1 };

// act(g) and its derivative. gelu(g) = g F(g) with F the normal distribution,
// whose error function is Abramowitz and Stegun's 7.1.26 (1.5e-7 off at most);
// its exponential is that of the derivative too.
template <int ACT>
__device__ __forceinline__ void activate(float g, float& a, float& da)
{
    if constexpr (ACT == ACT_SILU) {
        const float t = __builtin_amdgcn_rcpf(1.f + exp2_fast(-g * LOG2E));
        a = g * t;
        da = fmaf(a, 1.f - t, t);
    } else {
        const float e = exp2_fast(g * g * (-0.5f * LOG2E));
        const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f * 0.70710678f, fabsf(g), 1.f));
        const float p = fmaf(fmaf(fmaf(fmaf(1.061405429f, t, -1.453152027f), t, 1.421413741f), t, -0.284496736f), t, 0.254829592f);
        const float q = 0.5f * p * t * e;  // F(-|g|)
        const float f = g < 0.f ? q : 1.f - q;
        a = g * f;
        da = fmaf(g * e, 0.39894228f, f);
    }
}

// What becomes of a product's elements.
enum { TO_STORE = 0, TO_GATED = 1, TO_GRAD = 2, TO_PART = 3 };

struct Target {
    void* out[2];        // STORE: rows below `half` to [0], the others, less half, to [1]; GATED: h; GRAD: gg | gu
    int64_t ld[2];       // elements
    int64_t half;
    float* pre;          // GATED: out, or null; GRAD: in: [rows][2 n], g | u
    float* part;         // PART: [splits][rows][columns]
    int64_t m, n;        // of C; columns of one matrix of a pair
};

template <typename T, int ACT>
__device__ __forceinline__ void gated_one(const Target& o, int64_t row, int64_t col, float g, float u)
{
    float a, da;
    activate<ACT>(g, a, da);
    ((T*)o.out[0])[row * o.ld[0] + col] = (T)(a * u);
    if (o.pre) {
        o.pre[row * 2 * o.n + col] = g;
        o.pre[row * 2 * o.n + o.n + col] = u;
    }
}

template <typename T, int ACT>
__device__ __forceinline__ void grad_one(const Target& o, int64_t row, int64_t col, float gh)
{
    const float g = o.pre[row * 2 * o.n + col], u = o.pre[row * 2 * o.n + o.n + col];
    float a, da;
    activate<ACT>(g, a, da);
    T* p = (T*)o.out[0] + row * o.ld[0] + col;
    p[0] = (T)(gh * u * da);
    p[o.n] = (T)(gh * a);
}

template <typename T>
__device__ __forceinline__ void store_one(const Target& o, int64_t row, int64_t col, float v)
{
    const int which = row >= o.half;
    ((T*)o.out[which])[(which ? row - o.half : row) * o.ld[which] + col] = (T)v;
}

struct ProductArgs {
    Operand a, b;
    Target o;
    Walk walk;
    uint32_t mt, nt, per_split;  // tiles, and stages of a split
};

template <typename T, typename S, bool ATR, bool BTR, int TO, int ACT, bool PART>
__device__ __forceinline__ void ff_product(char* __restrict__ lds, const ProductArgs& p)
{
    constexpr bool PAIR = TO == TO_GATED;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id(), hi = lane >> 5;
    const uint32_t tiles = p.mt * p.nt, split = uniform(blockIdx.x / tiles);
    uint32_t mi, ni;
    tile_of(xcd_contiguous(blockIdx.x - split * tiles, tiles), p.mt, p.nt, mi, ni);
    const int64_t m0 = (int64_t)mi * S::BM, n0 = (int64_t)ni * (PAIR ? S::BN / 2 : S::BN);
    Walk w = p.walk;
    w.first = split * p.per_split;
    w.last = min(w.last, w.first + p.per_split);
    acc16 acc[S::MT][S::NT];
    TileProduct<T, S, ATR, BTR, PAIR>::run(lds, p.a, p.b, m0, n0, w, wave, acc);
    const int64_t row0 = m0 + wave / S::WN * (S::BM / S::WM);
    const int64_t col0 = n0 + wave % S::WN * (S::BN / S::WN / (PAIR ? 2 : 1)) + (lane & 31);
#pragma unroll
    for (int i = 0; i < S::MT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int64_t row = row0 + 32 * i + c_row(r, hi);
            if (row >= p.o.m) continue;
#pragma unroll
            for (int j = 0; j < S::NT; ++j) {
                if constexpr (PAIR) {
                    if (j & 1 || col0 >= p.o.n) continue;
                    if constexpr (PART) {
                        float* to = p.o.part + (split * p.o.m + row) * 2 * p.o.n + col0;
                        to[0] = acc[i][j][r];
                        to[p.o.n] = acc[i][j + 1][r];
                    } else {
                        gated_one<T, ACT>(p.o, row, col0, acc[i][j][r], acc[i][j + 1][r]);
                    }
                } else {
                    const int64_t col = col0 + 32 * j;
                    if (col >= p.o.n) continue;
                    if constexpr (PART) p.o.part[(split * p.o.m + row) * p.o.n + col] = acc[i][j][r];
                    else if constexpr (TO == TO_GRAD) grad_one<T, ACT>(p.o, row, col, acc[i][j][r]);
                    else store_one<T>(p.o, row, col, acc[i][j][r]);
                }
            }
        }
}

template <typename T, typename S, bool ATR, bool BTR, int TO, int ACT, bool PART>
__global__ __launch_bounds__(S::WAVES * 64, 2) void k_ff_product(const ProductArgs p)
{
    __shared__ alignas(16) char s_lds[TileProduct<T, S, ATR, BTR, TO == TO_GATED>::LDS];
    ff_product<T, S, ATR, BTR, TO, ACT, PART>(s_lds, p);
}

// The splits' sums, in order, and what becomes of them.
template <typename T, int TO, int ACT>
__global__ __launch_bounds__(256) void k_ff_join(const Target o, int32_t splits)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= o.m * o.n) return;
    const int64_t row = i / o.n, col = i - row * o.n, width = TO == TO_GATED ? 2 * o.n : o.n;
    float v = 0.f, u = 0.f;
    for (int s = 0; s < splits; ++s) {
        const float* p = o.part + (s * o.m + row) * width + col;
        v += p[0];
        if (TO == TO_GATED) u += p[o.n];
    }
    if constexpr (TO == TO_GATED) gated_one<T, ACT>(o, row, col, v, u);
    else if constexpr (TO == TO_GRAD) grad_one<T, ACT>(o, row, col, v);
    else store_one<T>(o, row, col, v);
}

// Operands along k (rows of 128 bytes a stage), both across, and few tiles.
using LargeK = TileShape<256, 256, 2, 4, 128, 2>;
using LargeT = TileShape<256, 256, 2, 4, 128, 2>;
using Small = TileShape<64, 128, 2, 2, 128, 3>;

// How a product of m x n over k is cut.
struct Cut {
    bool large;
    int32_t stages, splits, per_split;
    int64_t mt, nt;
};

static Cut cut_of(int64_t m, int64_t n, int64_t k, int segments, bool pair, bool across)
{
    Cut c;
    const int64_t wide = pair ? 2 * n : n, rows = across ? LargeT::BM : LargeK::BM;
    c.large = ((m + rows - 1) / rows) * ((wide + 255) / 256) >= 128;
    const int bm = c.large ? (int)rows : Small::BM, ke = (c.large ? (across ? LargeT::KB : LargeK::KB) : Small::KB) / 2;
    c.mt = (m + bm - 1) / bm;
    c.nt = (wide + (c.large ? 255 : 127)) / (c.large ? 256 : 128);
    c.stages = (int32_t)((k + ke - 1) / ke);
    const int64_t total = (int64_t)c.stages * segments, tiles = c.mt * c.nt;
    int64_t splits = std::max<int64_t>(1, std::min<int64_t>(512 / std::max<int64_t>(tiles, 1), total / 4));
    c.per_split = (int32_t)std::max<int64_t>(1, (total + splits - 1) / splits);
    c.splits = (int32_t)std::max<int64_t>(1, (total + c.per_split - 1) / c.per_split);
    return c;
}

static size_t part_bytes(const Cut& c, int64_t m, int64_t n, bool pair)
{
    return c.splits > 1 ? (size_t)c.splits * m * n * (pair ? 2 : 1) * 4 : 0;
}

template <typename T, bool ATR, bool BTR, int TO, int ACT>
static hipError_t product(const Operand& a, const Operand& b, Target o, int64_t k, int segments, float* part, hipStream_t s)
{
    using Large = std::conditional_t<ATR, LargeT, LargeK>;
    const Cut c = cut_of(o.m, o.n, k, segments, TO == TO_GATED, ATR);
    ProductArgs p;
    p.a = a;
    p.b = b;
    o.part = part;
    p.o = o;
    p.walk = {k, c.stages, 0, c.stages * segments};
    p.mt = (uint32_t)c.mt;
    p.nt = (uint32_t)c.nt;
    p.per_split = c.per_split;
    const dim3 grid((unsigned)(c.mt * c.nt * c.splits));
    if (c.splits > 1) {
        if (c.large) hipLaunchKernelGGL((k_ff_product<T, Large, ATR, BTR, TO, ACT, true>), grid, dim3(c.large ? 512 : 256), 0, s, p);
        else hipLaunchKernelGGL((k_ff_product<T, Small, ATR, BTR, TO, ACT, true>), grid, dim3(c.large ? 512 : 256), 0, s, p);
        hipLaunchKernelGGL((k_ff_join<T, TO, ACT>), dim3(grid_for((uint64_t)(o.m * o.n), 256)), dim3(256), 0, s, p.o, c.splits);
    } else {
        if (c.large) hipLaunchKernelGGL((k_ff_product<T, Large, ATR, BTR, TO, ACT, false>), grid, dim3(c.large ? 512 : 256), 0, s, p);
        else hipLaunchKernelGGL((k_ff_product<T, Small, ATR, BTR, TO, ACT, false>), grid, dim3(c.large ? 512 : 256), 0, s, p);
    }
    return hipGetLastError();
}

struct Sizes {
    int64_t rows, c, f, co;
};

static bool sizes_ok(const Sizes& z)
{
    return z.rows >= 0 && z.rows <= (1 << 24) && z.c >= 8 && z.f >= 8 && z.co >= 8 && z.c <= (1 << 17) && z.f <= (1 << 17) &&
           z.co <= (1 << 17) && z.c % 8 == 0 && z.f % 8 == 0 && z.co % 8 == 0;
}

// Whether every product's workgroups, of 256 threads, are below 2^32 threads.
static bool tiles_ok(const Sizes& z)
{
    const auto fits = [](const Cut& c) { return c.mt * c.nt < (1 << 23); };
    return fits(cut_of(z.rows, z.f, z.c, 1, true, false)) && fits(cut_of(z.rows, z.co, z.f, 1, false, false)) &&
           fits(cut_of(z.rows, z.c, z.f, 2, false, false)) && fits(cut_of(2 * z.f, z.c, z.rows, 1, false, true)) &&
           fits(cut_of(z.co, z.f, z.rows, 1, false, true));
}

static size_t fwd_bytes(const Sizes& z)
{
    return std::max(part_bytes(cut_of(z.rows, z.f, z.c, 1, true, false), z.rows, z.f, true),
                    part_bytes(cut_of(z.rows, z.co, z.f, 1, false, false), z.rows, z.co, false));
}

static size_t grad_bytes(const Sizes& z) { return ((size_t)z.rows * z.f * 2 * 2 + 255) / 256 * 256; }  // gg | gu

static size_t bwd_bytes(const Sizes& z)
{
    size_t part = part_bytes(cut_of(z.rows, z.f, z.co, 1, false, false), z.rows, z.f, false);
    part = std::max(part, part_bytes(cut_of(z.rows, z.c, z.f, 2, false, false), z.rows, z.c, false));
    part = std::max(part, part_bytes(cut_of(2 * z.f, z.c, z.rows, 1, false, true), 2 * z.f, z.c, false));
    return grad_bytes(z) + std::max(part, part_bytes(cut_of(z.co, z.f, z.rows, 1, false, true), z.co, z.f, false));
}

static Operand operand(const gs_matrix* m, int64_t rows) { return {{(const char*)m->data, nullptr}, {m->stride * 2, 0}, rows}; }

static Operand operand(const gs_matrix* m, const gs_matrix* second, int64_t rows)
{
    return {{(const char*)m->data, (const char*)second->data}, {m->stride * 2, second->stride * 2}, rows};
}

static Operand dense(const void* p, int64_t ld, int64_t rows) { return {{(const char*)p, nullptr}, {ld * 2, 0}, rows}; }

static Target target(void* out, int64_t ld, int64_t m, int64_t n, float* pre = nullptr)
{
    return {{out, nullptr}, {ld, 0}, m, pre, nullptr, m, n};
}

template <typename T, int ACT>
static hipError_t ff_fwd(const Sizes& z, const gs_matrix* x, const gs_matrix* wg, const gs_matrix* wu, const gs_matrix* wd,
                         void* h, float* pre, void* y, float* part, hipStream_t s)
{
    hipError_t e = product<T, false, false, TO_GATED, ACT>(operand(x, z.rows), operand(wg, wu, z.f),
                                                           target(h, z.f, z.rows, z.f, pre), z.c, 1, part, s);
    if (e == hipSuccess)
        e = product<T, false, false, TO_STORE, ACT_SILU>(dense(h, z.f, z.rows), operand(wd, z.co), target(y, z.co, z.rows, z.co),
                                                         z.f, 1, part, s);
    return e;
}

template <typename T, int ACT>
static hipError_t ff_bwd(const Sizes& z, const gs_matrix* gy, const gs_matrix* x, const gs_matrix* wg, const gs_matrix* wu,
                         const gs_matrix* wd, const void* h, const float* pre, void* gx, void* gwg, void* gwu, void* gwd,
                         void* ws, hipStream_t s)
{
    char* g = (char*)ws;  // gg | gu
    float* part = (float*)(g + grad_bytes(z));
    hipError_t e = product<T, false, true, TO_GRAD, ACT>(operand(gy, z.rows), operand(wd, z.f),
                                                         target(g, 2 * z.f, z.rows, z.f, (float*)pre), z.co, 1, part, s);
    if (e == hipSuccess && gx) {
        Operand a{{g, g + z.f * 2}, {z.f * 4, z.f * 4}, z.rows};
        e = product<T, false, true, TO_STORE, ACT_SILU>(a, operand(wg, wu, z.c), target(gx, z.c, z.rows, z.c), z.f, 2, part, s);
    }
    if (e == hipSuccess && gwg) {
        Target o = target(gwg, z.c, 2 * z.f, z.c);
        o.out[1] = gwu;
        o.ld[1] = z.c;
        o.half = z.f;
        e = product<T, true, true, TO_STORE, ACT_SILU>(dense(g, 2 * z.f, 2 * z.f), operand(x, z.c), o, z.rows, 1, part, s);
    }
    if (e == hipSuccess && gwd)
        e = product<T, true, true, TO_STORE, ACT_SILU>(operand(gy, z.co), dense(h, z.f, z.f), target(gwd, z.f, z.co, z.f), z.rows,
                                                       1, part, s);
    return e;
}

// Rows on 16 bytes, and those of a tile within 31 bits.
static bool ff_rows_ok(const gs_matrix* m)
{
    return ((uintptr_t)m->data & 15) == 0 && m->stride % 8 == 0 && m->stride >= 0 && m->stride < (1 << 21);
}

__global__ __launch_bounds__(256) void k_ff_zero(uint4* p, int64_t n)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = uint4{0, 0, 0, 0};
}

// Zeros over a matrix of a multiple of 8 16-bit elements.
static hipError_t ff_zero(void* p, int64_t elements, hipStream_t s)
{
    if (!p) return hipSuccess;
    hipLaunchKernelGGL(k_ff_zero, dim3(grid_for((uint64_t)elements / 8, 256)), dim3(256), 0, s, (uint4*)p, elements / 8);
    return hipGetLastError();
}

static bool given(const gs_matrix* m) { return m && m->data; }

}  // namespace gs

extern "C" {

size_t gs_gated_ff_fwd_workspace_bytes(int64_t rows, int32_t channels, int32_t hidden, int32_t channels_out)
{
    const gs::Sizes z{rows, channels, hidden, channels_out};
    return gs::sizes_ok(z) ? gs::fwd_bytes(z) : 0;
}

gs_status gs_gated_ff_fwd(const gs_matrix* x, const gs_matrix* w_gate, const gs_matrix* w_up, const gs_matrix* w_down,
                          int64_t rows, int32_t channels, int32_t hidden, int32_t channels_out, int32_t act, int32_t dtype,
                          void* h, float* pre, void* y, void* ws, size_t ws_bytes, void* stream)
{
    using namespace gs;
    const Sizes z{rows, channels, hidden, channels_out};
    if (!sizes_ok(z) || !dtype_ok(dtype) || (act != GS_SILU && act != GS_GELU)) return GS_ERR_INVALID_ARGUMENT;
    if (dtype == GS_F32 || !tiles_ok(z)) return GS_ERR_UNSUPPORTED;
    if (rows == 0) return GS_OK;
    if (!given(x) || !given(w_gate) || !given(w_up) || !given(w_down) || !h || !y) return GS_ERR_INVALID_ARGUMENT;
    const size_t need = fwd_bytes(z);
    if (need && (!ws || ((uintptr_t)ws & 15) || ws_bytes < need)) return GS_ERR_INVALID_ARGUMENT;
    if (!ff_rows_ok(x) || !ff_rows_ok(w_gate) || !ff_rows_ok(w_up) || !ff_rows_ok(w_down) || (((uintptr_t)h | (uintptr_t)y) & 15))
        return GS_ERR_UNSUPPORTED;
    const hipStream_t s = (hipStream_t)stream;
    const auto f = dtype == GS_F16 ? (act == GS_SILU ? ff_fwd<f16, ACT_SILU> : ff_fwd<f16, ACT_GELU>)
                                   : (act == GS_SILU ? ff_fwd<bf16, ACT_SILU> : ff_fwd<bf16, ACT_GELU>);
    return f(z, x, w_gate, w_up, w_down, h, pre, y, (float*)ws, s) == hipSuccess ? GS_OK : GS_ERR_HIP;
}

size_t gs_gated_ff_bwd_workspace_bytes(int64_t rows, int32_t channels, int32_t hidden, int32_t channels_out)
{
    const gs::Sizes z{rows, channels, hidden, channels_out};
    return gs::sizes_ok(z) ? gs::bwd_bytes(z) + 64 : 0;
}

gs_status gs_gated_ff_bwd(const gs_matrix* gy, const gs_matrix* x, const gs_matrix* w_gate, const gs_matrix* w_up,
                          const gs_matrix* w_down, const void* h, const float* pre, int64_t rows, int32_t channels,
                          int32_t hidden, int32_t channels_out, int32_t act, int32_t dtype, void* gx, void* gw_gate,
                          void* gw_up, void* gw_down, void* ws, size_t ws_bytes, void* stream)
{
    using namespace gs;
    const Sizes z{rows, channels, hidden, channels_out};
    if (!sizes_ok(z) || !dtype_ok(dtype) || (act != GS_SILU && act != GS_GELU) || !gw_gate != !gw_up)
        return GS_ERR_INVALID_ARGUMENT;
    if (dtype == GS_F32 || !tiles_ok(z)) return GS_ERR_UNSUPPORTED;
    if (!ws || ((uintptr_t)ws & 15) || ws_bytes < gs_gated_ff_bwd_workspace_bytes(rows, channels, hidden, channels_out))
        return GS_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)gx | (uintptr_t)gw_gate | (uintptr_t)gw_up | (uintptr_t)gw_down) & 15) return GS_ERR_UNSUPPORTED;
    const hipStream_t s = (hipStream_t)stream;
    if (rows == 0) {
        const int64_t n = (int64_t)hidden * channels;
        for (void* p : {gw_gate, gw_up})
            if (ff_zero(p, n, s) != hipSuccess) return GS_ERR_HIP;
        return ff_zero(gw_down, (int64_t)channels_out * hidden, s) == hipSuccess ? GS_OK : GS_ERR_HIP;
    }
    if (!given(gy) || !given(x) || !given(w_gate) || !given(w_up) || !given(w_down) || !h || !pre) return GS_ERR_INVALID_ARGUMENT;
    if (!ff_rows_ok(gy) || !ff_rows_ok(x) || !ff_rows_ok(w_gate) || !ff_rows_ok(w_up) || !ff_rows_ok(w_down) || ((uintptr_t)h & 15))
        return GS_ERR_UNSUPPORTED;
    const auto f = dtype == GS_F16 ? (act == GS_SILU ? ff_bwd<f16, ACT_SILU> : ff_bwd<f16, ACT_GELU>)
                                   : (act == GS_SILU ? ff_bwd<bf16, ACT_SILU> : ff_bwd<bf16, ACT_GELU>);
    return f(z, gy, x, w_gate, w_up, w_down, h, pre, gx, gw_gate, gw_up, gw_down, ws, s) == hipSuccess ? GS_OK : GS_ERR_HIP;
}

}  // extern "C"
