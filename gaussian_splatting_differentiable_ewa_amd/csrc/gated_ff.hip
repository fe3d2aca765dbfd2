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

// g and u as the forward pass keeps them for the backward pass: 16 bits of their
// fp32 in a plane each, and bits of both that follow in a third: 4 each with bf16
// (12 significant bits in all), 8 each with fp16 (16). Kept in the inputs' type
// alone, their roundings would add to those of gg and gu; kept whole, they are
// 8 bytes an element instead of 5 or 6, and both kernels that touch them wait
// for memory.
template <typename T>
struct Kept {
    static constexpr int MORE = std::is_same<T, bf16>::value ? 4 : 8;
    typedef std::conditional_t<MORE == 4, uint8_t, uint16_t> Low;
    static constexpr int BYTES = 4 + sizeof(Low);  // an element
    char* p;
    int64_t plane;  // elements
    __device__ __forceinline__ uint16_t* g(int64_t i) const { return (uint16_t*)p + i; }
    __device__ __forceinline__ uint16_t* u(int64_t i) const { return (uint16_t*)p + plane + i; }
    __device__ __forceinline__ Low* low(int64_t i) const { return (Low*)(p + 4 * plane) + i; }
    // Rounded to 16 + MORE bits, in the upper ones.
    static __device__ __forceinline__ uint32_t cut(float x)
    {
        const uint32_t b = __builtin_bit_cast(uint32_t, x) + (1u << (15 - MORE));
        return x != x ? 0x7fc00000u : b;
    }
    static __device__ __forceinline__ Low lows(uint32_t g, uint32_t u)
    {
        constexpr uint32_t M = (1u << MORE) - 1;
        return (Low)((g >> (16 - MORE) & M) | (u >> (16 - MORE) & M) << MORE);
    }
    static __device__ __forceinline__ float whole(uint32_t high, uint32_t low)
    {
        return __builtin_bit_cast(float, high << 16 | (low & ((1u << MORE) - 1)) << (16 - MORE));
    }
};

// What becomes of a product's elements.
enum { TO_STORE = 0, TO_GATED = 1, TO_GRAD = 2 };

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
    // h, and what is kept of g and u
    static __device__ __forceinline__ void gate(const float (&g)[4], const float (&u)[4], Vec<T, 4>& h, Vec<uint16_t, 4>& kg,
                                                Vec<uint16_t, 4>& ku, Vec<typename Kept<T>::Low, 4>& low)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float a, da;
            activate<ACT>(g[e], a, da);
            h.v[e] = (T)(a * u[e]);
            const uint32_t cg = Kept<T>::cut(g[e]), cu = Kept<T>::cut(u[e]);
            kg.v[e] = (uint16_t)(cg >> 16);
            ku.v[e] = (uint16_t)(cu >> 16);
            low.v[e] = Kept<T>::lows(cg, cu);
        }
    }
    // gg and gu from gh
    static __device__ __forceinline__ void grad(const float (&gh)[4], const Vec<uint16_t, 4>& kg, const Vec<uint16_t, 4>& ku,
                                                const Vec<typename Kept<T>::Low, 4>& low, Vec<T, 4>& gg, Vec<T, 4>& gu)
    {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float g = Kept<T>::whole(kg.v[e], low.v[e]), u = Kept<T>::whole(ku.v[e], low.v[e] >> Kept<T>::MORE);
            float a, da;
            activate<ACT>(g, a, da);
            gg.v[e] = (T)(gh[e] * u * da);
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

// The wave's rows from m0 + 32 i on and columns from n0 on, for each i, out of
// its accumulators through its scratch.
template <typename T, typename S, int TO, int ACT, bool PART>
__device__ __forceinline__ void finish(char* __restrict__ scratch, const Target& o, const acc16 (&acc)[S::MT][S::NT],
                                       int64_t m0, int64_t n0, int64_t split)
{
    const int lane = lane_id(), hi = lane >> 5;
    constexpr bool PAIR = TO == TO_GATED;
    constexpr int COLS = S::NT * 32 / (PAIR ? 2 : 1);
    const int64_t cols = o.n - n0 < COLS ? o.n - n0 : COLS;  // may be negative
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
            const Rows<W * sizeof(typename Kept<T>::Low) / 2> low{scratch + 96 * W};
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
                    Vec<uint16_t, 4> kg, ku;
                    Vec<typename Kept<T>::Low, 4> kl;
                    Four<T, ACT>::gate(vg, vu, vh, kg, ku, kl);
                    const int c = 32 * j + 8 * r + 4 * hi;
                    h.put(c * 2, vh);
                    if (o.kept) {
                        g.put(c * 2, kg);
                        u.put(c * 2, ku);
                        low.put(c * (int)sizeof(typename Kept<T>::Low), kl);
                    }
                }
            wait_lds();
            h.store((char*)((T*)o.out[0] + row0 * o.ld[0] + n0), o.ld[0] * 2, rows, cols * 2);
            if (o.kept) {
                const int64_t first = row0 * o.n + n0;
                g.store((char*)kept.g(first), o.n * 2, rows, cols * 2);
                u.store((char*)kept.u(first), o.n * 2, rows, cols * 2);
                low.store8((char*)kept.low(first), o.n * (int)sizeof(typename Kept<T>::Low), rows,
                           cols * (int)sizeof(typename Kept<T>::Low));
            }
        } else if constexpr (TO == TO_GRAD) {
            constexpr int W = COLS * 2;
            const Rows<W> g{scratch}, u{scratch + 32 * W};
            const Rows<W * sizeof(typename Kept<T>::Low) / 2> low{scratch + 64 * W};
            const Kept<T> kept{o.kept, o.m * o.n};
            const int64_t first = row0 * o.n + n0;
            wait_lds();
            g.load((const char*)kept.g(first), o.n * 2, rows, cols * 2);
            u.load((const char*)kept.u(first), o.n * 2, rows, cols * 2);
            low.load8((const char*)kept.low(first), o.n * (int)sizeof(typename Kept<T>::Low), rows,
                      cols * (int)sizeof(typename Kept<T>::Low));
            wait_lds();
#pragma unroll
            for (int j = 0; j < S::NT; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float gh[4];
                    four(j, r, gh);
                    const int c = 32 * j + 8 * r + 4 * hi;
                    Vec<T, 4> gg, gu;
                    Four<T, ACT>::grad(gh, g.template get<Vec<uint16_t, 4>>(c * 2), u.template get<Vec<uint16_t, 4>>(c * 2),
                                       low.template get<Vec<typename Kept<T>::Low, 4>>(c * (int)sizeof(typename Kept<T>::Low)),
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

template <typename T, typename S, bool ATR, bool BTR, int TO, int ACT, bool PART, bool TWO>
__device__ __forceinline__ void ff_product(char* __restrict__ lds, const ProductArgs& p)
{
    constexpr bool PAIR = TO == TO_GATED;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t tiles = p.mt * p.nt, split = uniform(blockIdx.x / tiles);
    uint32_t mi, ni;
    tile_of(xcd_contiguous(blockIdx.x - split * tiles, tiles), p.mt, p.nt, mi, ni);
    const int64_t m0 = (int64_t)mi * S::BM, n0 = (int64_t)ni * (PAIR ? S::BN / 2 : S::BN);
    Walk w = p.walk;
    w.first = split * p.per_split;
    w.last = min(w.last, w.first + p.per_split);
    acc16 acc[S::MT][S::NT];
    using Tiles = TileProduct<T, S, ATR, BTR, PAIR, TWO>;
    Tiles::run(lds, p.a, p.b, m0, n0, w, wave, acc);
    static_assert(Tiles::LDS / S::WAVES >= 32 * 64 * 4 * 2, "a wave's scratch");
    finish<T, S, TO, ACT, PART>(lds + wave * (Tiles::LDS / S::WAVES), p.o, acc, m0 + wave / S::WN * (S::BM / S::WM),
                                n0 + wave % S::WN * (S::BN / S::WN / (PAIR ? 2 : 1)), split);
}

template <typename T, typename S, bool ATR, bool BTR, int TO, int ACT, bool PART, bool TWO>
__global__ __launch_bounds__(S::WAVES * 64, S::PER_SIMD) void k_ff_product(const ProductArgs p)
{
    __shared__ alignas(16) char s_lds[TileProduct<T, S, ATR, BTR, TO == TO_GATED, TWO>::LDS];
    ff_product<T, S, ATR, BTR, TO, ACT, PART, TWO>(s_lds, p);
}

// The splits' sums, in order, and what becomes of them; four columns a thread.
template <typename T, int TO, int ACT>
__global__ __launch_bounds__(256) void k_ff_join(const Target o, int32_t splits)
{
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
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
    using Low4 = Vec<typename Kept<T>::Low, 4>;
    using High4 = Vec<uint16_t, 4>;
    const Kept<T> kept{o.kept, o.m * o.n};
    if constexpr (TO == TO_GATED) {
        Vec<T, 4> h;
        High4 kg, ku;
        Low4 low;
        Four<T, ACT>::gate(v, u, h, kg, ku, low);
        *(Vec<T, 4>*)((T*)o.out[0] + row * o.ld[0] + col) = h;
        if (o.kept) {
            *(High4*)kept.g(at) = kg;
            *(High4*)kept.u(at) = ku;
            *(Low4*)kept.low(at) = low;
        }
    } else if constexpr (TO == TO_GRAD) {
        Vec<T, 4> gg, gu;
        Four<T, ACT>::grad(v, *(const High4*)kept.g(at), *(const High4*)kept.u(at), *(const Low4*)kept.low(at), gg, gu);
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

// Few rows (16 at most): the weights are read once and bound it, so each wave
// takes them straight from memory to registers, 16 rows of them and the tokens
// beside them to a 16 x 16 tile of the result, and the waves of a workgroup
// share the sum over k, 64 elements in turn: a lane's two pieces of 16 bytes and
// its three neighbours' are 128 bytes of a row (the order of k inside a product
// is free as long as both operands have the same). Their sums meet in LDS.
// With PARTS = 2 a tile is 8 rows of the weights for 8 tokens, each twice, with
// the first and the second half of k: of the 16 x 16 results the two 8 x 8 count
// whose halves are the same. It makes twice the workgroups, for few columns.
constexpr int FEW = 16;

struct FewArgs {
    const char *x, *w[2];
    int64_t ld_x, ld[2];  // bytes
    Target o;
    int32_t k;
};

template <typename T, int TO, int ACT, int WAVES, int PARTS>
__global__ __launch_bounds__(WAVES * 64) void k_ff_few(const FewArgs p)
{
    constexpr int M = TO == TO_GATED ? 2 : 1, AHEAD = (WAVES < 16 ? 8 : 4) / M, SIDE = 16 / PARTS;
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
        Vec<uint16_t, 4> kg, ku;
        Vec<typename Kept<T>::Low, 4> low;
        Four<T, ACT>::gate(v, u, h, kg, ku, low);
        *(Vec<T, 4>*)((T*)p.o.out[0] + r * p.o.ld[0] + col) = h;
        if (p.o.kept) {
            const Kept<T> kept{p.o.kept, p.o.m * p.o.n};
            const int64_t at = r * p.o.n + col;
            *(Vec<uint16_t, 4>*)kept.g(at) = kg;
            *(Vec<uint16_t, 4>*)kept.u(at) = ku;
            *(Vec<typename Kept<T>::Low, 4>*)kept.low(at) = low;
        }
    } else {
        Vec<T, 4> t;
#pragma unroll
        for (int e = 0; e < 4; ++e) t.v[e] = (T)v[e];
        *(Vec<T, 4>*)((T*)p.o.out[0] + r * p.o.ld[0] + col) = t;
    }
}

// Waves to a workgroup: enough for the chip where there are few columns.
template <typename T, int TO, int ACT>
static hipError_t few(const Operand& a, const Operand& b, const Target& o, int64_t k, hipStream_t s)
{
    FewArgs p;
    p.x = a.data[0];
    p.ld_x = a.ld[0];
    for (int i = 0; i < 2; ++i) p.w[i] = b.data[i], p.ld[i] = b.ld[i];
    p.o = o;
    p.k = (int32_t)k;
    const auto launch = [&](auto waves, auto parts) {
        constexpr int W = decltype(waves)::value, P = decltype(parts)::value;
        hipLaunchKernelGGL((k_ff_few<T, TO, ACT, W, P>), dim3((unsigned)((o.n + 16 / P - 1) / (16 / P))), dim3(W * 64), 0, s, p);
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 8> eight;
    if (k <= 512) launch(four, one);
    else if (o.m <= 8 && o.n <= 4096) launch(eight, two);
    else launch(eight, one);
    return hipGetLastError();
}

// Many tiles, and few.
using Wide = TileShape<256, 256, 2, 4, 128, 2>;
using Small = TileShape<64, 128, 2, 2, 128, 3>;

// How a product of m x n over k is cut.
struct Cut {
    bool large;
    int32_t stages, splits, per_split;
    int64_t mt, nt;
};

template <typename S>
static Cut cut_as(bool large, int64_t m, int64_t wide, int64_t k, int segments, int64_t slots)
{
    Cut c;
    c.large = large;
    c.mt = (m + S::BM - 1) / S::BM;
    c.nt = (wide + S::BN - 1) / S::BN;
    c.stages = (int32_t)((k + S::KB / 2 - 1) / (S::KB / 2));
    const int64_t total = (int64_t)c.stages * segments, tiles = std::max<int64_t>(c.mt * c.nt, 1);
    const int64_t splits = std::max<int64_t>(1, std::min<int64_t>(slots / tiles, total / 4));
    c.per_split = (int32_t)std::max<int64_t>(1, (total + splits - 1) / splits);
    c.splits = (int32_t)std::max<int64_t>(1, (total + c.per_split - 1) / c.per_split);
    return c;
}

static Cut cut_of(int64_t m, int64_t n, int64_t k, int segments, int to)
{
    const int64_t wide = to == TO_GATED ? 2 * n : n;
    if (((m + 255) / 256) * ((wide + 255) / 256) < 128) return cut_as<Small>(false, m, wide, k, segments, 512);
    return cut_as<Wide>(true, m, wide, k, segments, 256);
}

static size_t part_bytes(const Cut& c, int64_t m, int64_t n, int to)
{
    return c.splits > 1 ? (size_t)c.splits * m * n * (to == TO_GATED ? 2 : 1) * 4 : 0;
}

template <typename T, bool ATR, bool BTR, int TO, int ACT, bool TWO = false>
static hipError_t product(const Operand& a, const Operand& b, Target o, int64_t k, float* part, hipStream_t s)
{
    constexpr int segments = TWO ? 2 : 1;
    const Cut c = cut_of(o.m, o.n, k, segments, TO);
    ProductArgs p;
    p.a = a;
    p.b = b;
    o.part = part;
    p.o = o;
    p.walk = {k, c.stages, 0, c.stages * segments};
    p.mt = (uint32_t)c.mt;
    p.nt = (uint32_t)c.nt;
    p.per_split = c.per_split;
    const dim3 grid((unsigned)(c.mt * c.nt * c.splits)), block((c.large ? Wide::WAVES : Small::WAVES) * 64);
    if (c.splits > 1) {
        if (c.large) hipLaunchKernelGGL((k_ff_product<T, Wide, ATR, BTR, TO, ACT, true, TWO>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((k_ff_product<T, Small, ATR, BTR, TO, ACT, true, TWO>), grid, block, 0, s, p);
        hipLaunchKernelGGL((k_ff_join<T, TO, ACT>), dim3(grid_for((uint64_t)(o.m * o.n / 4), 256)), dim3(256), 0, s, p.o, c.splits);
    } else {
        if (c.large) hipLaunchKernelGGL((k_ff_product<T, Wide, ATR, BTR, TO, ACT, false, TWO>), grid, block, 0, s, p);
        else hipLaunchKernelGGL((k_ff_product<T, Small, ATR, BTR, TO, ACT, false, TWO>), grid, block, 0, s, p);
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
    return fits(cut_of(z.rows, z.f, z.c, 1, TO_GATED)) && fits(cut_of(z.rows, z.co, z.f, 1, TO_STORE)) &&
           fits(cut_of(z.rows, z.f, z.co, 1, TO_GRAD)) && fits(cut_of(z.rows, z.c, z.f, 2, TO_STORE)) && fits(cut_of(2 * z.f, z.c, z.rows, 1, TO_STORE)) &&
           fits(cut_of(z.co, z.f, z.rows, 1, TO_STORE));
}

static size_t fwd_bytes(const Sizes& z)
{
    if (z.rows <= FEW) return 0;
    return std::max(part_bytes(cut_of(z.rows, z.f, z.c, 1, TO_GATED), z.rows, z.f, TO_GATED),
                    part_bytes(cut_of(z.rows, z.co, z.f, 1, TO_STORE), z.rows, z.co, TO_STORE));
}

static size_t grad_bytes(const Sizes& z) { return ((size_t)z.rows * z.f * 2 * 2 + 255) / 256 * 256; }  // gg | gu

static size_t bwd_bytes(const Sizes& z)
{
    size_t part = part_bytes(cut_of(z.rows, z.f, z.co, 1, TO_GRAD), z.rows, z.f, TO_GRAD);
    part = std::max(part, part_bytes(cut_of(z.rows, z.c, z.f, 2, TO_STORE), z.rows, z.c, TO_STORE));
    part = std::max(part, part_bytes(cut_of(2 * z.f, z.c, z.rows, 1, TO_STORE), 2 * z.f, z.c, TO_STORE));
    return grad_bytes(z) + std::max(part, part_bytes(cut_of(z.co, z.f, z.rows, 1, TO_STORE), z.co, z.f, TO_STORE));
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
    hipError_t e = product<T, false, false, TO_GATED, ACT>(operand(x, z.rows), operand(wg, wu, z.f),
                                                           target(h, z.f, z.rows, z.f, kept), z.c, part, s);
    if (e == hipSuccess)
        e = product<T, false, false, TO_STORE, ACT_SILU>(dense(h, z.f, z.rows), operand(wd, z.co), target(y, z.co, z.rows, z.co),
                                                         z.f, part, s);
    return e;
}

template <typename T, int ACT>
static hipError_t ff_bwd(const Sizes& z, const gs_matrix* gy, const gs_matrix* x, const gs_matrix* wg, const gs_matrix* wu,
                         const gs_matrix* wd, const void* h, const void* kept, void* gx, void* gwg, void* gwu, void* gwd,
                         void* ws, hipStream_t s)
{
    char* g = (char*)ws;  // gg | gu
    float* part = (float*)(g + grad_bytes(z));
    hipError_t e = product<T, false, true, TO_GRAD, ACT>(operand(gy, z.rows), operand(wd, z.f),
                                                         target(g, 2 * z.f, z.rows, z.f, (void*)kept), z.co, part, s);
    if (e == hipSuccess && gx) {
        Operand a{{g, g + z.f * 2}, {z.f * 4, z.f * 4}, z.rows};
        e = product<T, false, true, TO_STORE, ACT_SILU, true>(a, operand(wg, wu, z.c), target(gx, z.c, z.rows, z.c), z.f, part, s);
    }
    if (e == hipSuccess && gwg) {
        Target o = target(gwg, z.c, 2 * z.f, z.c);
        o.out[1] = gwu;
        o.ld[1] = z.c;
        o.half = z.f;
        e = product<T, true, true, TO_STORE, ACT_SILU>(dense(g, 2 * z.f, 2 * z.f), operand(x, z.c), o, z.rows, part, s);
    }
    if (e == hipSuccess && gwd)
        e = product<T, true, true, TO_STORE, ACT_SILU>(operand(gy, z.co), dense(h, z.f, z.f), target(gwd, z.f, z.co, z.f), z.rows,
                                                       part, s);
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
    if (!ff_rows_ok(x) || !ff_rows_ok(w_gate) || !ff_rows_ok(w_up) || !ff_rows_ok(w_down) || (((uintptr_t)h | (uintptr_t)kept | (uintptr_t)y) & 15))
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
    if (!ff_rows_ok(gy) || !ff_rows_ok(x) || !ff_rows_ok(w_gate) || !ff_rows_ok(w_up) || !ff_rows_ok(w_down) || (((uintptr_t)h | (uintptr_t)kept) & 15))
        return GS_ERR_UNSUPPORTED;
    const auto f = dtype == GS_F16 ? (act == GS_SILU ? ff_bwd<f16, ACT_SILU> : ff_bwd<f16, ACT_GELU>)
                                   : (act == GS_SILU ? ff_bwd<bf16, ACT_SILU> : ff_bwd<bf16, ACT_GELU>);
    return f(z, gy, x, w_gate, w_up, w_down, h, kept, gx, gw_gate, gw_up, gw_down, ws, s) == hipSuccess ? GS_OK : GS_ERR_HIP;
}

}  // extern "C"
