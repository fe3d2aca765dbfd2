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
// which the matrix unit takes them.
#include "gated_plan.h"
#include "product.h"

namespace gs {

enum { ACT_SILU = 0, ACT_GELU = 1 };

// act(g) and its derivative. gelu(g) = g F(g) with F the normal distribution. For
// g < 0, with x = |g| / sqrt 2 and t = 1 / (1 + 0.33 x), F = t P(t) exp(-x^2) / 2: P, of
// degree 7, is fitted to erfc(x) exp(x^2) / t over x of 0 to 9.6 for the least largest
// error relative to it, 8.2e-8, so a closing gate keeps its digits: 5e-7 off with the
// roundings at g = -1, 2e-6 at -6 and 8e-6 at -12, where the exponent's argument
// is 104. (Abramowitz and Stegun's 7.1.26, three terms shorter, is 5e-4 off at -4 and
// 1e-2 at -8; the largest training step is 0.4 % faster with it.) The exponential is
// that of the derivative too.
template <int ACT>
__device__ __forceinline__ void activate(float g, float& a, float& da)
{
    if constexpr (ACT == ACT_SILU) {
        const float t = __builtin_amdgcn_rcpf(1.f + exp2_fast(-g * LOG2E));
        a = g * t;
        da = fmaf(a, 1.f - t, t);
    } else {
        const float e = exp2_fast(g * g * (-0.5f * LOG2E));
        const float t = __builtin_amdgcn_rcpf(fmaf(0.33f * 0.70710678f, fabsf(g), 1.f));
        float p = fmaf(-0.135929227f, t, 0.462690145f);
        p = fmaf(fmaf(fmaf(p, t, -0.355442464f), t, 0.412545085f), t, 0.0450086333f);
        p = fmaf(fmaf(fmaf(p, t, 0.201924488f), t, 0.182837129f), t, 0.186366126f);
        const float q = 0.5f * p * t * e;  // F(-|g|)
        const float f = g < 0.f ? q : 1.f - q;
        a = g * f;
        da = fmaf(g * e, 0.39894228f, f);
    }
}

// g and u as the forward pass keeps them for the backward pass: 16 bits of their
// fp32 in a plane each, and bits of both that follow in a third: 4 each with bf16
// (12 significant bits in all), 8 each with fp16 (16). Kept in the inputs' type
// alone, their roundings would add to those of gg and gu; kept whole, they are
// 8 bytes an element instead of 5 or 6, and both kernels that touch them wait
// for memory.
template <typename T>
struct Kept {
    static constexpr int MORE = std::is_same<T, bf16>::value ? 4 : 8;
    static constexpr int LOW = 2 * MORE / 8, BYTES = 4 + LOW;  // of the third plane, and in all, an element
    typedef std::conditional_t<LOW == 1, uint32_t, uint2> Low4;  // of four elements
    char* p;
    int64_t plane;  // elements
    __device__ __forceinline__ uint16_t* g(int64_t i) const { return (uint16_t*)p + i; }
    __device__ __forceinline__ uint16_t* u(int64_t i) const { return (uint16_t*)p + plane + i; }
    __device__ __forceinline__ char* low(int64_t i) const { return p + 4 * plane + i * LOW; }
    // Rounded to 16 + MORE bits, in the upper ones.
    static __device__ __forceinline__ uint32_t cut(float x)
    {
        const uint32_t b = __builtin_bit_cast(uint32_t, x) + (1u << (15 - MORE));
        return x != x ? 0x7fc00000u : b;
    }
    // Four elements' bits by v_perm_b32, which takes any four of eight bytes: 3 to 5
    // instructions an element less than with shifts and masks, where a tile's 65536
    // elements pass the CU's 64 lanes with no product beside them.
    static __device__ __forceinline__ uint32_t upper(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302); }
    static __device__ __forceinline__ void pack(const float (&g)[4], const float (&u)[4], uint2& kg, uint2& ku, Low4& low)
    {
        uint32_t a[4], b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = cut(g[e]), b[e] = cut(u[e]);
        kg = {upper(a[0], a[1]), upper(a[2], a[3])};
        ku = {upper(b[0], b[1]), upper(b[2], b[3])};
        const auto second = [](uint32_t x, uint32_t y, uint32_t to) { return __builtin_amdgcn_perm(y, x, to); };
        constexpr uint32_t LOWER = 0x0c0c0501, HIGHER = 0x05010c0c;  // both second bytes, to either half
        if constexpr (LOW == 1) {  // a byte an element: g's bits above u's
            const uint32_t x = second(a[0], a[1], LOWER) | second(a[2], a[3], HIGHER);
            const uint32_t y = second(b[0], b[1], LOWER) | second(b[2], b[3], HIGHER);
            low = (x & 0xf0f0f0f0u) | (y >> 4 & 0x0f0f0f0fu);
        } else {  // two: g's, u's
            low = {second(a[0], b[0], LOWER) | second(a[1], b[1], HIGHER), second(a[2], b[2], LOWER) | second(a[3], b[3], HIGHER)};
        }
    }
    static __device__ __forceinline__ void unpack(uint2 kg, uint2 ku, Low4 low, float (&g)[4], float (&u)[4])
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t high = e % 2 ? 0x0706000cu : 0x0504000cu;  // 16 bits, a byte to come, and zeros
            const uint32_t hg = e < 2 ? kg.x : kg.y, hu = e < 2 ? ku.x : ku.y;
            if constexpr (LOW == 1) {
                g[e] = __builtin_bit_cast(float, __builtin_amdgcn_perm(hg, low & 0xf0f0f0f0u, high | e << 8));
                u[e] = __builtin_bit_cast(float, __builtin_amdgcn_perm(hu, low << 4 & 0xf0f0f0f0u, high | e << 8));
            } else {
                const uint32_t w = e < 2 ? low.x : low.y;
                g[e] = __builtin_bit_cast(float, __builtin_amdgcn_perm(hg, w, high | 2 * (e % 2) << 8));
                u[e] = __builtin_bit_cast(float, __builtin_amdgcn_perm(hu, w, high | (2 * (e % 2) + 1) << 8));
            }
        }
    }
};

struct Target {
    void* out[2];   // STORE: rows below `half` to [0], the others, less half, to [1]; GATED: h; GRAD: gg | gu
    int64_t ld[2];  // elements
    int64_t half;
    char* kept;     // GATED: out, or null; GRAD: in
    float* part;    // of a product in splits: [splits][rows][columns]
    int64_t m, n;   // of C; columns of one matrix of a pair
};

template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T v[N];
};

// Four columns from `col` on of one row.
template <typename T, int ACT>
struct Four {
    using Low4 = typename Kept<T>::Low4;
    // h, and what is kept of g and u
    static __device__ __forceinline__ void gate(const float (&g)[4], const float (&u)[4], Vec<T, 4>& h, uint2& kg, uint2& ku, Low4& low)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, da;
            activate<ACT>(g[e], a, da);
            h.v[e] = (T)(a * u[e]);
        }
        Kept<T>::pack(g, u, kg, ku, low);
    }
    // gg and gu from gh
    static __device__ __forceinline__ void grad(const float (&gh)[4], uint2 kg, uint2 ku, Low4 low, Vec<T, 4>& gg, Vec<T, 4>& gu)
    {
        float g[4], u[4];
        Kept<T>::unpack(kg, ku, low, g, u);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, da;
            activate<ACT>(g[e], a, da);
            gg.v[e] = (T)(gh[e] * u[e] * da);
            gu.v[e] = (T)(gh[e] * a);
        }
    }
};

struct ProductArgs {
    Operand a, b;
    Target o;
    Walk walk;
    uint32_t mt, nt, per_split;  // tiles, and stages of a split
};

// Of 32 rows of COLS columns, what the forward pass kept, on its way from memory
// to a scratch. It is read 32 rows ahead; with the packing above that took
// 32640 x 2048 x 8192 from 1378 to 1300 us.
template <typename T, int COLS>
struct Held {
    uint4 g[COLS / 16], u[COLS / 16];
    uint2 low[COLS * Kept<T>::LOW / 16];
    __device__ __forceinline__ void fetch(const Target& o, int64_t row0, int64_t n0, int64_t cols)
    {
        const Kept<T> kept{o.kept, o.m * o.n};
        const int64_t first = row0 * o.n + n0, rows = o.m - row0;
        Rows<COLS * 2>::fetch(g, (const char*)kept.g(first), o.n * 2, rows, cols * 2);
        Rows<COLS * 2>::fetch(u, (const char*)kept.u(first), o.n * 2, rows, cols * 2);
        Rows<COLS * Kept<T>::LOW>::fetch(low, kept.low(first), o.n * Kept<T>::LOW, rows, cols * Kept<T>::LOW);
    }
};

// The wave's rows from m0 + 32 i on and columns from n0 on, for each i, out of
// its accumulators through its scratch.
template <typename T, typename S, int TO, int ACT, bool PART>
__device__ __forceinline__ void finish(char* scratch, const Target& o, const acc16 (&acc)[S::MT][S::NT],
                                       int64_t m0, int64_t n0, int64_t split)
{
    const int lane = lane_id(), hi = lane >> 5;
    constexpr bool PAIR = TO == TO_GATED;
    constexpr int COLS = S::NT * 32 / (PAIR ? 2 : 1);
    const int64_t cols = o.n - n0 < COLS ? o.n - n0 : COLS;  // may be negative
    Held<T, COLS> held;
    if constexpr (TO == TO_GRAD && !PART) held.fetch(o, m0, n0, cols);
#pragma unroll
    for (int i = 0; i < S::MT; ++i) {
        const int64_t row0 = m0 + 32 * i, rows = o.m - row0;
        const auto four = [&](int j, int r, float (&v)[4]) __attribute__((always_inline)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * r + e];
        };
        if constexpr (PART) {
            const Rows<128> at{scratch};
            const int64_t width = PAIR ? 2 * o.n : o.n;
#pragma unroll
            for (int j = 0; j < S::NT; ++j) {
                wait_lds();
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    Vec<float, 4> v;
                    four(j, r, v.v);
                    at.put(32 * r + 16 * hi, v);
                }
                wait_lds();
                const int c = j % (COLS / 32) * 32;
                float* to = o.part + (split * o.m + row0) * width + n0 + c + (PAIR && j >= S::NT / 2 ? o.n : 0);
                at.store((char*)to, width * 4, rows, (cols - c) * 4);
            }
        } else if constexpr (TO == TO_GATED) {
            constexpr int W = COLS * 2;
            const Rows<W> h{scratch}, g{scratch + 32 * W}, u{scratch + 64 * W};
            const Rows<COLS * Kept<T>::LOW> low{scratch + 96 * W};
            const Kept<T> kept{o.kept, o.m * o.n};
            wait_lds();
#pragma unroll
            for (int j = 0; j < S::NT / 2; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float vg[4], vu[4];
                    four(j, r, vg);
                    four(j + S::NT / 2, r, vu);
                    Vec<T, 4> vh;
                    uint2 kg, ku;
                    typename Kept<T>::Low4 kl;
                    Four<T, ACT>::gate(vg, vu, vh, kg, ku, kl);
                    const int c = 32 * j + 8 * r + 4 * hi;
                    h.put(c * 2, vh);
                    if (o.kept) {
                        g.put(c * 2, kg);
                        u.put(c * 2, ku);
                        low.put(c * Kept<T>::LOW, kl);
                    }
                }
            wait_lds();
            h.store((char*)((T*)o.out[0] + row0 * o.ld[0] + n0), o.ld[0] * 2, rows, cols * 2);
            if (o.kept) {
                const int64_t first = row0 * o.n + n0;
                g.store((char*)kept.g(first), o.n * 2, rows, cols * 2);
                u.store((char*)kept.u(first), o.n * 2, rows, cols * 2);
                low.store8((char*)kept.low(first), o.n * Kept<T>::LOW, rows,
                           cols * Kept<T>::LOW);
            }
        } else if constexpr (TO == TO_GRAD) {
            constexpr int W = COLS * 2;
            const Rows<W> g{scratch}, u{scratch + 32 * W};
            const Rows<COLS * Kept<T>::LOW> low{scratch + 64 * W};
            wait_lds();
            g.put_all(held.g);
            u.put_all(held.u);
            low.put_all(held.low);
            wait_lds();
            if (i + 1 < S::MT) held.fetch(o, row0 + 32, n0, cols);  // while these are worked on
#pragma unroll
            for (int j = 0; j < S::NT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float gh[4];
                    four(j, r, gh);
                    const int c = 32 * j + 8 * r + 4 * hi;
                    Vec<T, 4> gg, gu;
                    Four<T, ACT>::grad(gh, g.template get<uint2>(c * 2), u.template get<uint2>(c * 2),
                                       low.template get<typename Kept<T>::Low4>(c * Kept<T>::LOW),
                                       gg, gu);
                    g.put(c * 2, gg);  // where its own were read
                    u.put(c * 2, gu);
                }
            wait_lds();
            T* to = (T*)o.out[0] + row0 * o.ld[0] + n0;
            g.store((char*)to, o.ld[0] * 2, rows, cols * 2);
            u.store((char*)(to + o.n), o.ld[0] * 2, rows, cols * 2);
        } else {
            constexpr int W = COLS * 2;
            const Rows<W> at{scratch};
            wait_lds();
#pragma unroll
            for (int j = 0; j < S::NT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float v[4];
                    four(j, r, v);
                    Vec<T, 4> t;
#pragma unroll
                    for (int e = 0; e < 4; ++e) t.v[e] = (T)v[e];
                    at.put(64 * j + 16 * r + 8 * hi, t);
                }
            wait_lds();
            // 32 rows lie on one side of `half`, a multiple of 8, or on both
            const int64_t below = o.half - row0;
            if (below > 0) at.store((char*)((T*)o.out[0] + row0 * o.ld[0] + n0), o.ld[0] * 2, below < rows ? below : rows, cols * 2);
            if (below < 32)
                at.store((char*)((T*)o.out[1] + (row0 - o.half) * o.ld[1] + n0), o.ld[1] * 2, rows, cols * 2, below);
        }
    }
}

// Block `id` of a product's.
template <typename T, typename S, bool ATR, bool BTR, int TO, int ACT, bool TWO>
__device__ __forceinline__ void ff_product(char* lds, const ProductArgs& p, uint32_t id)
{
    constexpr bool PAIR = TO == TO_GATED;
    const int all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), group = all / S::WAVES, wave = all % S::WAVES;
    const uint32_t tiles = p.mt * p.nt, split = uniform(id / tiles);
    uint32_t mi, ni;
    tile_of(xcd_contiguous(id - split * tiles, tiles), p.mt, p.nt, mi, ni);
    const int64_t m0 = (int64_t)mi * S::BM, n0 = (int64_t)ni * (PAIR ? S::BN / 2 : S::BN);
    Walk w = p.walk;
    w.first = split * p.per_split;
    w.last = min(w.last, w.first + (int)p.per_split);
    acc16 acc[S::MT][S::NT];
    using Tiles = TileProduct<T, S, ATR, BTR, PAIR, TWO>;
    Tiles::run(lds, p.a, p.b, m0, n0, w, group, wave, acc);
    if (group > 0) return;
    char* scratch = lds + wave * Tiles::SCRATCH;
    const int64_t m = m0 + wave / S::WN * (S::BM / S::WM), n = n0 + wave % S::WN * (S::BN / S::WN / (PAIR ? 2 : 1));
    // h, g, u and what they keep beyond 16 bits, or a row of 32 sums at a time
    static_assert(Tiles::SCRATCH >= std::max(S::BN / S::WN / (PAIR ? 2 : 1) * 2 * 32 * 4, 32 * 128), "a wave's scratch");
    if (p.o.part) finish<T, S, TO, ACT, true>(scratch, p.o, acc, m, n, split);
    else finish<T, S, TO, ACT, false>(scratch, p.o, acc, m, n, 0);
}

template <typename T, typename S, bool ATR, bool BTR, int TO, int ACT>
__global__ __launch_bounds__(S::THREADS, S::PER_SIMD) void k_ff_product(const ProductArgs p)
{
    __shared__ alignas(16) char s_lds[TileProduct<T, S, ATR, BTR, TO == TO_GATED>::LDS];
    ff_product<T, S, ATR, BTR, TO, ACT, false>(s_lds, p, blockIdx.x);
}

// gx, the two projections' gradients and the last one's: blocks of each in turn.
struct BackArgs {
    ProductArgs p[3];
    uint32_t blocks[3];
};

template <typename T, typename S>
__global__ __launch_bounds__(S::THREADS, S::PER_SIMD) void k_ff_back(const BackArgs b)
{
    __shared__ alignas(16) char s_lds[TileProduct<T, S, true, true, false>::LDS];
    uint32_t id = blockIdx.x;
    if (id < b.blocks[0]) {
        ff_product<T, S, false, true, TO_STORE, ACT_SILU, true>(s_lds, b.p[0], id);
        return;
    }
    id -= b.blocks[0];
    const int which = id < b.blocks[1] ? 1 : 2;
    ff_product<T, S, true, true, TO_STORE, ACT_SILU, false>(s_lds, b.p[which], which == 1 ? id : id - b.blocks[1]);
}

// The splits' sums, in order, and what becomes of them; four columns a thread.
template <typename T, int TO, int ACT>
__device__ __forceinline__ void ff_join(const Target& o, int32_t splits, uint32_t id)
{
    const int64_t at = ((int64_t)id * 256 + threadIdx.x) * 4;
    if (at >= o.m * o.n) return;
    const int64_t row = at / o.n, col = at - row * o.n, width = TO == TO_GATED ? 2 * o.n : o.n;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const float* p = o.part + (s * o.m + row) * width + col;
        const Vec<float, 4> x = *(const Vec<float, 4>*)p;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += x.v[e];
        if (TO == TO_GATED) {
            const Vec<float, 4> y = *(const Vec<float, 4>*)(p + o.n);
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] += y.v[e];
        }
    }
    using Low4 = typename Kept<T>::Low4;
    const Kept<T> kept{o.kept, o.m * o.n};
    if constexpr (TO == TO_GATED) {
        Vec<T, 4> h;
        uint2 kg, ku;
        Low4 low;
        Four<T, ACT>::gate(v, u, h, kg, ku, low);
        *(Vec<T, 4>*)((T*)o.out[0] + row * o.ld[0] + col) = h;
        if (o.kept) {
            *(uint2*)kept.g(at) = kg;
            *(uint2*)kept.u(at) = ku;
            *(Low4*)kept.low(at) = low;
        }
    } else if constexpr (TO == TO_GRAD) {
        Vec<T, 4> gg, gu;
        Four<T, ACT>::grad(v, *(const uint2*)kept.g(at), *(const uint2*)kept.u(at), *(const Low4*)kept.low(at), gg, gu);
        T* to = (T*)o.out[0] + row * o.ld[0] + col;
        *(Vec<T, 4>*)to = gg;
        *(Vec<T, 4>*)(to + o.n) = gu;
    } else {
        const int which = row >= o.half;
        Vec<T, 4> t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t.v[e] = (T)v[e];
        *(Vec<T, 4>*)((T*)o.out[which] + (which ? row - o.half : row) * o.ld[which] + col) = t;
    }
}

template <typename T, int TO, int ACT>
__global__ __launch_bounds__(256) void k_ff_join(const Target o, int32_t splits)
{
    ff_join<T, TO, ACT>(o, splits, blockIdx.x);
}

struct JoinArgs {
    Target o[3];
    int32_t splits[3];
    uint32_t blocks[3];
};

template <typename T>
__global__ __launch_bounds__(256) void k_ff_joins(const JoinArgs j)
{
    uint32_t id = blockIdx.x;
    int which = 0;
    while (which < 2 && id >= j.blocks[which]) id -= j.blocks[which++];
    ff_join<T, TO_STORE, ACT_SILU>(j.o[which], j.splits[which], id);
}

// Few rows (16 at most): the weights are read once and bound it (one row, 2048 x
// 8192: 67 MB in 13.0 us and 34 MB in 8.4, 5.2 and 4.0 TB/s), so each wave
// takes them straight from memory to registers, 16 rows of them and the tokens
// beside them to a 16 x 16 tile of the result, and the waves of a workgroup
// share the sum over k, 64 elements in turn: a lane's two pieces of 16 bytes and
// its three neighbours' are 128 bytes of a row (the order of k inside a product
// is free as long as both operands have the same). Their sums meet in LDS.
// With PARTS = 2 a tile is 8 rows of the weights for 8 tokens, each twice, with
// the first and the second half of k: of the 16 x 16 results the two 8 x 8 count
// whose halves are the same. It makes twice the workgroups, for up to 8 rows and
// few columns: one row, 2048 columns, k 8192: 8.4 us against 12.2, k 2048: 4.5
// against 5.4 (8 rows); 8192 columns, k 2048: 10.2 against 9.4.
// The tiles below take as long at 16 rows of 2048 x 8192 (33 us with their
// joins' launches, as here) and longer at fewer and smaller: 16 rows of 1024 x
// 4096 19.2 against 16.7, 12 of 520 x 1368 15.8 against 8.2.
constexpr int FEW = 16, FEW_WAVES = 8, NARROW = 4096;

struct FewArgs {
    const char *x, *w[2];
    int64_t ld_x, ld[2];  // bytes
    Target o;
    int32_t k;
};

template <typename T, int TO, int ACT, int PARTS>
__global__ __launch_bounds__(FEW_WAVES * 64) void k_ff_few(const FewArgs p)
{
    constexpr int WAVES = FEW_WAVES, M = TO == TO_GATED ? 2 : 1, AHEAD = 8 / M, SIDE = 16 / PARTS;
    typedef typename Mma<T>::v8 V;
    __shared__ float4v s_sum[WAVES][M][64];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane % SIDE, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * SIDE;
    const int rows = (int)p.o.m, part = PARTS > 1 ? lane >> 3 & 1 : 0;
    const int span = PARTS > 1 ? (p.k / 2 + 63) / 64 * 64 : p.k;  // of k a part has
    const int first = part * span + q * 16, end = part * span + span < p.k ? part * span + span : p.k;
    const char* x = p.x + (r < rows ? r : rows - 1) * p.ld_x;
    const int64_t row = n0 + r < p.o.n ? n0 + r : p.o.n - 1;
    const char* w[M];
#pragma unroll
    for (int i = 0; i < M; ++i) w[i] = p.w[i] + row * p.ld[i];
    float4v acc[M];
#pragma unroll
    for (int i = 0; i < M; ++i) acc[i] = float4v{0.f, 0.f, 0.f, 0.f};
    const auto load = [&](const char* from, int k, int half) __attribute__((always_inline)) {
        const int at = first + k + half * 8;
        V v{};
        if (at < end) v = *(const V*)(from + at * 2);
        return v;
    };
    for (int k0 = wave * 64; k0 < span; k0 += WAVES * 64 * AHEAD) {
        V vx[AHEAD][2], vw[AHEAD][M][2];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < M; ++i) vw[a][i][h] = load(w[i], k0 + a * WAVES * 64, h);
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) vx[a][h] = load(x, k0 + a * WAVES * 64, h);
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < M; ++i) acc[i] = mma16<T>(vw[a][i][h], vx[a][h], acc[i]);
    }
#pragma unroll
    for (int i = 0; i < M; ++i) s_sum[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave > 0) return;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < WAVES; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] += s_sum[i][0][lane][e];
            if (M > 1) u[e] += s_sum[i][M - 1][lane][e];
            if (PARTS > 1) {  // token r's second half, rows 8 on of the tile: 8 lanes and two quarters further
                const int other = (lane + 40) % 64;
                v[e] += s_sum[i][0][other][e];
                if (M > 1) u[e] += s_sum[i][M - 1][other][e];
            }
        }
    // of the result a lane holds token r, columns 4 q on
    const int64_t col = n0 + 4 * q;
    if (r >= rows || col >= p.o.n || part > 0 || 4 * q >= SIDE) return;
    if constexpr (TO == TO_GATED) {
        Vec<T, 4> h;
        uint2 kg, ku;
        typename Kept<T>::Low4 low;
        Four<T, ACT>::gate(v, u, h, kg, ku, low);
        *(Vec<T, 4>*)((T*)p.o.out[0] + r * p.o.ld[0] + col) = h;
        if (p.o.kept) {
            const Kept<T> kept{p.o.kept, p.o.m * p.o.n};
            const int64_t at = r * p.o.n + col;
            *(uint2*)kept.g(at) = kg;
            *(uint2*)kept.u(at) = ku;
            *(typename Kept<T>::Low4*)kept.low(at) = low;
        }
    } else {
        Vec<T, 4> t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t.v[e] = (T)v[e];
        *(Vec<T, 4>*)((T*)p.o.out[0] + r * p.o.ld[0] + col) = t;
    }
}

template <typename T, int TO, int ACT>
static hipError_t few(const Operand& a, const Operand& b, const Target& o, int64_t k, hipStream_t s)
{
    FewArgs p;
    p.x = a.data[0];
    p.ld_x = a.ld[0];
    for (int i = 0; i < 2; ++i) p.w[i] = b.data[i], p.ld[i] = b.ld[i];
    p.o = o;
    p.k = (int32_t)k;
    const auto blocks = [&](int64_t side) { return dim3((unsigned)((o.n + side - 1) / side)); };
    if (o.m <= 8 && o.n <= NARROW) hipLaunchKernelGGL((k_ff_few<T, TO, ACT, 2>), blocks(8), dim3(FEW_WAVES * 64), 0, s, p);
    else hipLaunchKernelGGL((k_ff_few<T, TO, ACT, 1>), blocks(16), dim3(FEW_WAVES * 64), 0, s, p);
    return hipGetLastError();
}

// The tiles. Wide's matrix instructions take 72 to 79 % of the cycles of y and of
// the backward's three products, 58 to 61 % with h's epilogue and 47 to 53 % with
// that of gg and gu, at clocks that fall to 1.3 to 1.75 GHz: 32640 x 8192 x 2048 in
// 857 to 865 us (1270 TFLOP/s; the library's own product 1526), the three products of
// the backward pass in 4080 to 4220 (1300, across k too; the library 1119 and 1243), and
// both projections with h and what is kept, 1.9 GB, in 2010 to 2090 (1050 to 1090). Of more
// stages or smaller ones, two workgroups of 256 x 128 on a CU, fetches to L2 ahead and wave
// priorities none was faster (865 against 899 to 1031).
// Smaller ones make more workgroups, and their groups of waves, which
// share the sum over k, fill the CU. Two groups of Small leave room for a second
// workgroup on the CU; four did not, and cost 1.2 us more a launch: 256 x 1024 x
// 1024 took 7.4 us either way, 1024 x 1024 x 1024 8.0 against 8.2 us, 4096 x 1024
// x 1024 29 against 21 us, 256 x 512 x 64 7.3 against 6.2 us.
using Wide = TileShape<256, 256, 2, 4, 128, 2>;
using Mid = TileShape<128, 128, 2, 2, 128, 2, 2>;
using Small = TileShape<64, 64, 2, 2, 128, 2, 2>;
using SmallPair = TileShape<64, 64, 2, 1, 128, 2, 2>;
static_assert(Small::BM == SIDE[SMALL] && Mid::BM == SIDE[MID] && Wide::BM == SIDE[WIDE] && Small::KG == GROUPS[SMALL] &&
                  Mid::KG == GROUPS[MID] && Wide::KG == GROUPS[WIDE],
              "the plan's tiles");

static ProductArgs args_of(const Operand& a, const Operand& b, const Target& o, int64_t k, int segments, const Cut& c, float* part)
{
    ProductArgs p;
    p.a = a;
    p.b = b;
    p.o = o;
    p.o.part = c.splits > 1 ? part : nullptr;
    p.walk = {k, c.stages, 0, c.stages * segments};
    p.mt = (uint32_t)c.mt;
    p.nt = (uint32_t)c.nt;
    p.per_split = (uint32_t)c.per_split;
    return p;
}

template <typename T, bool BTR, int TO, int ACT>
static hipError_t product(const Operand& a, const Operand& b, const Target& o, int64_t k, float* part, hipStream_t s)
{
    using Least = std::conditional_t<TO == TO_GATED, SmallPair, Small>;
    int shape;
    const Cut c = cut_of(o.m, o.n, k, TO, &shape);
    const ProductArgs p = args_of(a, b, o, k, 1, c, part);
    const dim3 grid((unsigned)c.blocks);
    if (shape == WIDE) hipLaunchKernelGGL((k_ff_product<T, Wide, false, BTR, TO, ACT>), grid, dim3(Wide::THREADS), 0, s, p);
    else if (shape == MID) hipLaunchKernelGGL((k_ff_product<T, Mid, false, BTR, TO, ACT>), grid, dim3(Mid::THREADS), 0, s, p);
    else hipLaunchKernelGGL((k_ff_product<T, Least, false, BTR, TO, ACT>), grid, dim3(Least::THREADS), 0, s, p);
    if (c.splits > 1)
        hipLaunchKernelGGL((k_ff_join<T, TO, ACT>), dim3(grid_for((uint64_t)(o.m * o.n / 4), 256)), dim3(256), 0, s, p.o, c.splits);
    return hipGetLastError();
}

static size_t fwd_bytes(const Sizes& z)
{
    if (z.rows <= FEW) return 0;
    int shape;
    return std::max(part_bytes(cut_of(z.rows, z.f, z.c, TO_GATED, &shape), z.rows, z.f, TO_GATED),
                    part_bytes(cut_of(z.rows, z.co, z.f, TO_STORE, &shape), z.rows, z.co, TO_STORE));
}

static size_t grad_bytes(const Sizes& z) { return ((size_t)z.rows * z.f * 2 * 2 + 255) / 256 * 256; }  // gg | gu

static size_t bwd_bytes(const Sizes& z)
{
    int shape;
    const Back b = back_of(z);
    size_t back = 0;
    for (int i = 0; i < 3; ++i) back += part_bytes(b.c[i], b.m[i], b.n[i], TO_STORE);
    return grad_bytes(z) + std::max(part_bytes(cut_of(z.rows, z.f, z.co, TO_GRAD, &shape), z.rows, z.f, TO_GRAD), back);
}

static Operand operand(const gs_matrix* m, int64_t rows) { return {{(const char*)m->data, nullptr}, {m->stride * 2, 0}, rows}; }

static Operand operand(const gs_matrix* m, const gs_matrix* second, int64_t rows)
{
    return {{(const char*)m->data, (const char*)second->data}, {m->stride * 2, second->stride * 2}, rows};
}

static Operand dense(const void* p, int64_t ld, int64_t rows) { return {{(const char*)p, nullptr}, {ld * 2, 0}, rows}; }

static Target target(void* out, int64_t ld, int64_t m, int64_t n, void* kept = nullptr)
{
    return {{out, nullptr}, {ld, 0}, m, (char*)kept, nullptr, m, n};
}

template <typename T, int ACT>
static hipError_t ff_fwd(const Sizes& z, const gs_matrix* x, const gs_matrix* wg, const gs_matrix* wu, const gs_matrix* wd,
                         void* h, void* kept, void* y, float* part, hipStream_t s)
{
    if (z.rows <= FEW) {
        const hipError_t e = few<T, TO_GATED, ACT>(operand(x, z.rows), operand(wg, wu, z.f), target(h, z.f, z.rows, z.f, kept), z.c, s);
        if (e != hipSuccess) return e;
        return few<T, TO_STORE, ACT_SILU>(dense(h, z.f, z.rows), operand(wd, z.co), target(y, z.co, z.rows, z.co), z.f, s);
    }
    const hipError_t e = product<T, false, TO_GATED, ACT>(operand(x, z.rows), operand(wg, wu, z.f),
                                                          target(h, z.f, z.rows, z.f, kept), z.c, part, s);
    if (e != hipSuccess) return e;
    return product<T, false, TO_STORE, ACT_SILU>(dense(h, z.f, z.rows), operand(wd, z.co), target(y, z.co, z.rows, z.co), z.f, part,
                                                 s);
}

template <typename T, int ACT>
static hipError_t ff_bwd(const Sizes& z, const gs_matrix* gy, const gs_matrix* x, const gs_matrix* wg, const gs_matrix* wu,
                         const gs_matrix* wd, const void* h, const void* kept, void* gx, void* gwg, void* gwu, void* gwd,
                         void* ws, hipStream_t s)
{
    char* g = (char*)ws;  // gg | gu
    float* part = (float*)(g + grad_bytes(z));
    const hipError_t e = product<T, true, TO_GRAD, ACT>(operand(gy, z.rows), operand(wd, z.f),
                                                        target(g, 2 * z.f, z.rows, z.f, (void*)kept), z.co, part, s);
    if (e != hipSuccess) return e;
    const Back b = back_of(z);
    const Operand gg{{g, g + z.f * 2}, {z.f * 4, z.f * 4}, z.rows};
    Target o[3] = {target(gx, z.c, z.rows, z.c), target(gwg, z.c, 2 * z.f, z.c), target(gwd, z.f, z.co, z.f)};
    o[1].out[1] = gwu;
    o[1].ld[1] = z.c;
    o[1].half = z.f;
    BackArgs p{};
    JoinArgs j{};
    for (int i = 0, joins = 0; i < 3; ++i) {
        if (!o[i].out[0]) continue;  // not wanted: no blocks
        p.p[i] = i == 0   ? args_of(gg, operand(wg, wu, z.c), o[0], z.f, 2, b.c[0], part)
                 : i == 1 ? args_of(dense(g, 2 * z.f, 2 * z.f), operand(x, z.c), o[1], z.rows, 1, b.c[1], part)
                          : args_of(operand(gy, z.co), dense(h, z.f, z.f), o[2], z.rows, 1, b.c[2], part);
        p.blocks[i] = (uint32_t)b.c[i].blocks;
        if (b.c[i].splits == 1) continue;
        part += part_bytes(b.c[i], b.m[i], b.n[i], TO_STORE) / 4;
        j.o[joins] = p.p[i].o;
        j.splits[joins] = b.c[i].splits;
        j.blocks[joins++] = grid_for((uint64_t)(b.m[i] * b.n[i] / 4), 256);
    }
    const dim3 grid(p.blocks[0] + p.blocks[1] + p.blocks[2]);
    if (grid.x == 0) return hipSuccess;
    if (b.shape == WIDE) hipLaunchKernelGGL((k_ff_back<T, Wide>), grid, dim3(Wide::THREADS), 0, s, p);
    else if (b.shape == MID) hipLaunchKernelGGL((k_ff_back<T, Mid>), grid, dim3(Mid::THREADS), 0, s, p);
    else hipLaunchKernelGGL((k_ff_back<T, Small>), grid, dim3(Small::THREADS), 0, s, p);
    if (j.blocks[0])
        hipLaunchKernelGGL((k_ff_joins<T>), dim3(j.blocks[0] + j.blocks[1] + j.blocks[2]), dim3(256), 0, s, j);
    return hipGetLastError();
}

// Rows on 16 bytes, those of a tile within 31 bits; rows that are one, or apart:
// what ends the last row ends every one behind it.
static bool ff_rows_ok(const gs_matrix* m, int64_t columns)
{
    return ((uintptr_t)m->data & 15) == 0 && m->stride % 8 == 0 && (m->stride == 0 || m->stride >= columns) && m->stride < (1 << 21);
}

// The same where sums run over the rows: those of one row for all would not end,
// and zeros of the other operand do not cancel an infinity.
static bool ff_rows_apart(const gs_matrix* m, int64_t columns) { return ff_rows_ok(m, columns) && m->stride != 0; }

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

size_t gs_gated_ff_kept_bytes(int64_t rows, int32_t hidden, int32_t dtype)
{
    using namespace gs;
    if (!sizes_ok({rows, 8, hidden, 8}) || (dtype != GS_F16 && dtype != GS_BF16)) return 0;
    return (size_t)rows * hidden * (dtype == GS_BF16 ? Kept<bf16>::BYTES : Kept<f16>::BYTES);
}

size_t gs_gated_ff_fwd_workspace_bytes(int64_t rows, int32_t channels, int32_t hidden, int32_t channels_out)
{
    const gs::Sizes z{rows, channels, hidden, channels_out};
    return gs::sizes_ok(z) ? gs::fwd_bytes(z) : 0;
}

gs_status gs_gated_ff_fwd(const gs_matrix* x, const gs_matrix* w_gate, const gs_matrix* w_up, const gs_matrix* w_down,
                          int64_t rows, int32_t channels, int32_t hidden, int32_t channels_out, int32_t act, int32_t dtype,
                          void* h, void* kept, void* y, void* ws, size_t ws_bytes, void* stream)
{
    using namespace gs;
    const Sizes z{rows, channels, hidden, channels_out};
    if (!sizes_ok(z) || !dtype_ok(dtype) || (act != GS_SILU && act != GS_GELU)) return GS_ERR_INVALID_ARGUMENT;
    if (dtype == GS_F32 || !tiles_ok(z)) return GS_ERR_UNSUPPORTED;
    if (rows == 0) return GS_OK;
    if (!given(x) || !given(w_gate) || !given(w_up) || !given(w_down) || !h || !y) return GS_ERR_INVALID_ARGUMENT;
    const size_t need = fwd_bytes(z);
    if (need && (!ws || ((uintptr_t)ws & 15) || ws_bytes < need)) return GS_ERR_INVALID_ARGUMENT;
    if (!ff_rows_ok(x, channels) || !ff_rows_ok(w_gate, channels) || !ff_rows_ok(w_up, channels) || !ff_rows_ok(w_down, hidden) ||
        (((uintptr_t)h | (uintptr_t)kept | (uintptr_t)y) & 15))
        return GS_ERR_UNSUPPORTED;
    const hipStream_t s = (hipStream_t)stream;
    const auto f = dtype == GS_F16 ? (act == GS_SILU ? ff_fwd<f16, ACT_SILU> : ff_fwd<f16, ACT_GELU>)
                                   : (act == GS_SILU ? ff_fwd<bf16, ACT_SILU> : ff_fwd<bf16, ACT_GELU>);
    return f(z, x, w_gate, w_up, w_down, h, kept, y, (float*)ws, s) == hipSuccess ? GS_OK : GS_ERR_HIP;
}

size_t gs_gated_ff_bwd_workspace_bytes(int64_t rows, int32_t channels, int32_t hidden, int32_t channels_out)
{
    const gs::Sizes z{rows, channels, hidden, channels_out};
    return gs::sizes_ok(z) ? gs::bwd_bytes(z) + 64 : 0;
}

gs_status gs_gated_ff_bwd(const gs_matrix* gy, const gs_matrix* x, const gs_matrix* w_gate, const gs_matrix* w_up,
                          const gs_matrix* w_down, const void* h, const void* kept, int64_t rows, int32_t channels,
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
    if (!given(gy) || !given(x) || !given(w_gate) || !given(w_up) || !given(w_down) || !h || !kept) return GS_ERR_INVALID_ARGUMENT;
    if (!ff_rows_apart(gy, channels_out) || !ff_rows_apart(x, channels) || !ff_rows_apart(w_gate, channels) ||
        !ff_rows_apart(w_up, channels) || !ff_rows_apart(w_down, hidden) || (((uintptr_t)h | (uintptr_t)kept) & 15))
        return GS_ERR_UNSUPPORTED;
    const auto f = dtype == GS_F16 ? (act == GS_SILU ? ff_bwd<f16, ACT_SILU> : ff_bwd<f16, ACT_GELU>)
                                   : (act == GS_SILU ? ff_bwd<bf16, ACT_SILU> : ff_bwd<bf16, ACT_GELU>);
    return f(z, gy, x, w_gate, w_up, w_down, h, kept, gx, gw_gate, gw_up, gw_down, ws, s) == hipSuccess ? GS_OK : GS_ERR_HIP;
}

}  // extern "C"
