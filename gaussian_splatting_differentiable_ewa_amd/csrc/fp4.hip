// gs_quantise_fp4, gs_dequantise_fp4 and gs_linear_fp4: microscaled 4-bit
// floating point, blocks of 32 values along a row that share a power of two.
//
// The matrix unit takes such values as they are, with the blocks' exponents
// beside them, at four times the rate of 16-bit ones: a product's tiles are the
// 16-bit ones of product.h, four times as long in k.
#include "product.h"

namespace gs {

constexpr int FP4_BLOCK = 32;

// The power of two a block's byte stands for (255: NaN).
__device__ __forceinline__ float power_of(uint32_t e)
{
    return __builtin_bit_cast(float, e == 0 ? 0x00400000u : (e == 255 ? 0x7fc00000u : e << 23));
}

// The byte of a block whose largest magnitude has these bits: its exponent less
// that of 4, so that it lies in 4 .. 8 (6 is the largest of the grid; what is
// over it rounds down). Infinities and NaN give 255, and a block of NaN.
__device__ __forceinline__ uint32_t byte_of(uint32_t bits)
{
    const uint32_t e = bits >> 23;
    return e == 255 ? 255 : (e > 2 ? e - 2 : 0);
}

// Eight values to codes, value i in bits 4 i; halves go to even codes.
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8], float power)
{
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], power, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], power, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], power, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], power, 3);
    return c;
}

__device__ __forceinline__ uint32_t largest_bits(const float (&v)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7fffffffu);
    return m;
}

// The largest over the four lanes of a block.
__device__ __forceinline__ uint32_t quad_max(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, false));  // quad_perm 1,0,3,2
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, false));  // quad_perm 2,3,0,1
}

// A thread's place: eight values at column c of row r0 + k step, k = 0, 1, ...
// Rows are dealt to `lanes` threads (a multiple of 4) or to several passes of
// 256 of them.
struct Eights {
    int64_t row, step;
    int c, stride;
    bool on;
    __device__ __forceinline__ explicit Eights(int channels)
    {
        const int lanes = channels / 8, t = threadIdx.x;
        const int per = lanes < 256 ? 256 / lanes : 1;
        const int r = lanes < 256 ? t / lanes : 0;
        on = r < per;
        row = (int64_t)blockIdx.x * per + r;
        step = (int64_t)gridDim.x * per;
        c = (lanes < 256 ? t - r * lanes : t) * 8;
        stride = 256 * 8;
    }
};

// Bound by HBM: a lane takes 16 or 32 bytes and gives 4, four lanes a block.
// 32640 x 2048 bf16: 28 to 33 us, 169 MB at 5.1 to 6.0 TB/s (rows that the writes
// of a moment ago left in the cache help), and the way back 26 us; four blocks in
// flight a thread took 40.
template <typename T>
__global__ __launch_bounds__(256) void k_fp4_quantise(const T* __restrict__ x, int64_t stride, uint8_t* __restrict__ codes,
                                                      uint8_t* __restrict__ scales, int64_t rows, int32_t channels,
                                                      int32_t scale_bytes)
{
    const Eights at(channels);
    if (!at.on) return;
    for (int64_t r = at.row; r < rows; r += at.step)
        for (int c = at.c; c < channels; c += at.stride) {
            float v[8];
            load_f32<T, 8>(x + r * stride + c, v);
            const uint32_t e = byte_of(quad_max(largest_bits(v)));
            *(uint32_t*)(codes + r * (channels / 2) + c / 2) = codes_of(v, power_of(e));
            if (c % FP4_BLOCK == 0) {
                const int b = c / FP4_BLOCK;
                scales[r * scale_bytes + b] = (uint8_t)e;
                if (c + FP4_BLOCK == channels)  // the bytes a row is filled up with
                    for (int i = b + 1; i < scale_bytes; ++i) scales[r * scale_bytes + i] = 0;
            }
        }
}

template <typename T>
__global__ __launch_bounds__(256) void k_fp4_dequantise(const uint8_t* __restrict__ codes, int64_t stride,
                                                        const uint8_t* __restrict__ scales, int64_t scale_stride,
                                                        T* __restrict__ out, int64_t rows, int32_t channels)
{
    typedef float float2v __attribute__((ext_vector_type(2)));
    const Eights at(channels);
    if (!at.on) return;
    for (int64_t r = at.row; r < rows; r += at.step)
        for (int c = at.c; c < channels; c += at.stride) {
            const uint32_t w = *(const uint32_t*)(codes + r * stride + c / 2);
            const float p = power_of(scales[r * scale_stride + c / FP4_BLOCK]);
            const float2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 1);
            const float2v d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 2), e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.f, 3);
            const float v[8] = {a[0] * p, a[1] * p, b[0] * p, b[1] * p, d[0] * p, d[1] * p, e[0] * p, e[1] * p};
            store_f32<T, 8>(out + r * channels + c, v);
        }
}

// A product's tiles: 32640 x 2048 x 8192 in 375 to 437 us, 2.5 to 2.9 PFLOP/s, where
// the 16-bit product takes 865. A step of the matrix unit lasts 32 cycles for 8 KB
// of operands; its instructions take 35 % of the cycles (at 1.97 GHz), the reads
// from LDS 33 %, 38 % of those in conflicts of banks: neither fills the time, and
// what keeps them from running beside each other is not found. 128 x 128 elements a workgroup, two to a CU, took 531; scales straight from memory to
// registers 618 (they share the address path with the tiles' loads).
struct FourArgs {
    Operand a, b;  // [0]: codes, [1]: scales
    Walk walk;
    void* y;
    int64_t m, n;
    uint32_t mt, nt;
};

using FourTile = TileShape<256, 256, 2, 4, 64, 4>;
using FourMid = TileShape<128, 128, 2, 2, 64, 4>;
using FourSmall = TileShape<64, 64, 2, 2, 64, 4>;

template <typename T, typename S>
__device__ __forceinline__ void four_product(char* lds, const FourArgs& p)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id(), hi = lane >> 5;
    uint32_t mi, ni;
    tile_of(xcd_contiguous(blockIdx.x, gridDim.x), p.mt, p.nt, mi, ni);
    const int64_t m0 = (int64_t)mi * S::BM, n0 = (int64_t)ni * S::BN;
    acc16 acc[S::MT][S::NT];
    TileProduct<fp4, S, false, false, false>::run(lds, p.a, p.b, m0, n0, p.walk, 0, wave, acc);
    // out through a scratch of the wave's own: whole rows, or where those do not lie on 16 bytes their elements
    using Tiles = TileProduct<fp4, S, false, false, false>;
    constexpr int SIZE = sizeof(T), PER = SIZE == 2 && S::NT > 1 ? 2 : 1, W = 32 * SIZE * PER;  // matrix tiles to a row of scratch
    static_assert(S::NT % PER == 0 && Tiles::SCRATCH >= 32 * W, "a wave's scratch");
    const Rows<W> at{lds + wave * (Tiles::SCRATCH)};
    const int64_t col0 = n0 + wave % S::WN * (S::BN / S::WN);
    const bool whole = p.n * SIZE % 16 == 0 && ((uintptr_t)p.y & 15) == 0;
#pragma unroll
    for (int i = 0; i < S::MT; ++i) {
        const int64_t row0 = m0 + wave / S::WN * (S::BM / S::WM) + 32 * i;
#pragma unroll
        for (int j = 0; j < S::NT; j += PER) {
            wait_lds();
#pragma unroll
            for (int q = 0; q < PER; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    struct alignas(4 * SIZE) {
                        T v[4];
                    } t;
#pragma unroll
                    for (int e = 0; e < 4; ++e) t.v[e] = (T)acc[i][j + q][4 * r + e];
                    at.put((32 * q + 8 * r + 4 * hi) * SIZE, t);
                }
            wait_lds();
            const int64_t col = col0 + 32 * j;
            char* to = (char*)((T*)p.y + row0 * p.n + col);
            if (whole) at.store(to, p.n * SIZE, p.m - row0, (p.n - col) * SIZE);
            else at.template store_as<std::conditional_t<SIZE == 2, uint16_t, uint32_t>>(to, p.n * SIZE, p.m - row0, (p.n - col) * SIZE, 0);
        }
    }
}

template <typename T, typename S>
__global__ __launch_bounds__(S::THREADS, 2) void k_fp4_product(const FourArgs p)
{
    __shared__ alignas(16) char s_lds[TileProduct<fp4, S, false, false, false>::LDS];
    four_product<T, S>(s_lds, p);
}

// Few rows (16 at most): one launch, bound by its latency (one row, 2048 to 8192:
// 9 MB in 5.7 us; quantised first, 1.6 us, and by the tiles above, 6.8 us; 16 rows
// 8.4 us against 2.5 and 6.6). A wave takes 16 rows of the weights and the
// tokens straight to registers, 128 values of each a step, a lane one block of
// 32 of either with its scale; it quantises the tokens' blocks itself (every
// workgroup does, which costs less than a launch before it). The waves of a
// workgroup share the sum, and theirs meet in LDS.
constexpr int FOUR_FEW = 16, FEW_WAVES = 8;

template <typename T>
__global__ __launch_bounds__(FEW_WAVES * 64) void k_fp4_few(const FourArgs p, const T* __restrict__ x, int64_t stride_x)
{
    typedef int v8i __attribute__((ext_vector_type(8)));
    __shared__ float4v s_sum[FEW_WAVES][64];
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, row = n0 + r < p.n ? n0 + r : p.n - 1;
    const int rows = (int)p.m, blocks = (int)p.walk.k / 8;
    const uint4* codes = (const uint4*)(p.b.data[0] + row * p.b.ld[0]);
    const uint8_t* scales = (const uint8_t*)p.b.data[1] + row * p.b.ld[1];
    const T* mine = x + (r < rows ? r : rows - 1) * stride_x;
    float4v acc = {0.f, 0.f, 0.f, 0.f};
    for (int b = wave * 4 + q; b < (blocks + 3) / 4 * 4; b += FEW_WAVES * 4) {
        v8i w = {}, t = {};
        int sw = 0, st = 0;
        if (b < blocks) {
            const uint4 c = codes[b];
            sw = scales[b];
            float v[4][8];
            uint32_t most = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                load_f32<T, 8>(mine + b * FP4_BLOCK + i * 8, v[i]);
                most = max(most, largest_bits(v[i]));
            }
            st = (int)byte_of(most);
            const float power = power_of(st);
            w[0] = c.x, w[1] = c.y, w[2] = c.z, w[3] = c.w;
#pragma unroll
            for (int i = 0; i < 4; ++i) t[i] = (int)codes_of(v[i], power);
        }
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, t, acc, 4, 4, 0, sw, 0, st);
    }
    s_sum[wave][lane] = acc;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 1; i < FEW_WAVES; ++i) acc += s_sum[i][lane];
    // of the result a lane holds token r, columns 4 q on
    if (r >= rows) return;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (n0 + 4 * q + e < p.n) ((T*)p.y)[r * p.n + n0 + 4 * q + e] = (T)acc[e];
}

template <typename T>
static hipError_t few_as(const FourArgs& p, const gs_matrix* x, hipStream_t s)
{
    hipLaunchKernelGGL((k_fp4_few<T>), dim3((unsigned)((p.n + 15) / 16)), dim3(FEW_WAVES * 64), 0, s, p, (const T*)x->data, x->stride);
    return hipGetLastError();
}

static int64_t scale_bytes_of(int32_t channels) { return (channels + 127) / 128 * 4; }

static unsigned eights_grid(int64_t rows, int32_t channels)
{
    const int64_t lanes = channels / 8, per = lanes < 256 ? 256 / lanes : 1;
    return (unsigned)std::min<int64_t>((rows + per - 1) / per, 8192);
}

template <typename T>
static hipError_t quantise(const void* x, int64_t stride, void* codes, void* scales, int64_t rows, int32_t channels, hipStream_t s)
{
    hipLaunchKernelGGL((k_fp4_quantise<T>), dim3(eights_grid(rows, channels)), dim3(256), 0, s, (const T*)x, stride,
                       (uint8_t*)codes, (uint8_t*)scales, rows, channels, (int32_t)scale_bytes_of(channels));
    return hipGetLastError();
}

static hipError_t quantise_as(int32_t dtype, const gs_matrix* x, void* codes, void* scales, int64_t rows, int32_t channels,
                              hipStream_t s)
{
    return dtype == GS_F32   ? quantise<float>(x->data, x->stride, codes, scales, rows, channels, s)
           : dtype == GS_F16 ? quantise<f16>(x->data, x->stride, codes, scales, rows, channels, s)
                             : quantise<bf16>(x->data, x->stride, codes, scales, rows, channels, s);
}

template <typename T>
static hipError_t dequantise(const gs_matrix* codes, const gs_matrix* scales, void* out, int64_t rows, int32_t channels,
                             hipStream_t s)
{
    hipLaunchKernelGGL((k_fp4_dequantise<T>), dim3(eights_grid(rows, channels)), dim3(256), 0, s, (const uint8_t*)codes->data,
                       codes->stride, (const uint8_t*)scales->data, scales->stride, (T*)out, rows, channels);
    return hipGetLastError();
}

template <typename T, typename S>
static hipError_t product_by(FourArgs& p, hipStream_t s)
{
    p.mt = (uint32_t)((p.m + S::BM - 1) / S::BM);
    p.nt = (uint32_t)((p.n + S::BN - 1) / S::BN);
    hipLaunchKernelGGL((k_fp4_product<T, S>), dim3(p.mt * p.nt), dim3(S::THREADS), 0, s, p);
    return hipGetLastError();
}

// The largest tiles that leave few CUs idle. With 192 tiles of 256 (6120 x 2048 x
// 2048) 23.5 us against 27.5 of 128, with 128 (4096 x 2048 x 2048) 21.3 against
// 20.0; with 232 of 128 (3600 x 1056 x 1000) 10.6 against 12.5 of 64, with 128
// (1024 x 2048 x 2048) 11.4 against 9.6.
template <typename T>
static hipError_t product_as(FourArgs& p, hipStream_t s)
{
    const auto tiles = [&](int64_t side) { return ((p.m + side - 1) / side) * ((p.n + side - 1) / side); };
    if (tiles(256) >= 192) return product_by<T, FourTile>(p, s);
    if (tiles(128) >= 160) return product_by<T, FourMid>(p, s);
    return product_by<T, FourSmall>(p, s);
}

static bool four_sizes_ok(int64_t rows, int32_t channels)
{
    return rows >= 0 && rows <= (1 << 24) && channels >= FP4_BLOCK && channels <= (1 << 17) && channels % FP4_BLOCK == 0;
}

// Rows on `align` bytes, those of a tile within 31 bits; rows that are one, or
// apart (`columns` of `unit` bytes each).
static bool four_rows_ok(const gs_matrix* m, int64_t columns, int unit, int align)
{
    return (uintptr_t)m->data % align == 0 && (m->stride == 0 || m->stride >= columns) && m->stride < (1 << 21) &&
           m->stride * unit % align == 0;
}

}  // namespace gs

extern "C" {

gs_status gs_quantise_fp4(const gs_matrix* x, int64_t rows, int32_t channels, int32_t dtype, void* codes, void* scales,
                          void* stream)
{
    using namespace gs;
    if (!four_sizes_ok(rows, channels) || !dtype_ok(dtype)) return GS_ERR_INVALID_ARGUMENT;
    if (rows == 0) return GS_OK;
    if (!x || !x->data || !codes || !scales) return GS_ERR_INVALID_ARGUMENT;
    if (!four_rows_ok(x, channels, elem_bytes(dtype), 16) || ((uintptr_t)codes & 15) || ((uintptr_t)scales & 3)) return GS_ERR_UNSUPPORTED;
    return quantise_as(dtype, x, codes, scales, rows, channels, (hipStream_t)stream) == hipSuccess ? GS_OK : GS_ERR_HIP;
}

gs_status gs_dequantise_fp4(const gs_matrix* codes, const gs_matrix* scales, int64_t rows, int32_t channels, int32_t dtype,
                            void* out, void* stream)
{
    using namespace gs;
    if (!four_sizes_ok(rows, channels) || !dtype_ok(dtype)) return GS_ERR_INVALID_ARGUMENT;
    if (rows == 0) return GS_OK;
    if (!codes || !codes->data || !scales || !scales->data || !out) return GS_ERR_INVALID_ARGUMENT;
    if (!four_rows_ok(codes, channels / 2, 1, 16) || !four_rows_ok(scales, scale_bytes_of(channels), 1, 4) || ((uintptr_t)out & 15)) return GS_ERR_UNSUPPORTED;
    const hipStream_t s = (hipStream_t)stream;
    const auto f = dtype == GS_F32 ? dequantise<float> : (dtype == GS_F16 ? dequantise<f16> : dequantise<bf16>);
    return f(codes, scales, out, rows, channels, s) == hipSuccess ? GS_OK : GS_ERR_HIP;
}

size_t gs_linear_fp4_workspace_bytes(int64_t rows, int32_t channels, int32_t out)
{
    using namespace gs;
    if (!four_sizes_ok(rows, channels) || out < 1 || out > (1 << 17) || rows <= FOUR_FEW) return 0;
    return ((size_t)rows * (channels / 2) + 15) / 16 * 16 + (size_t)rows * scale_bytes_of(channels) + 64;
}

gs_status gs_linear_fp4(const gs_matrix* x, const gs_matrix* codes, const gs_matrix* scales, int64_t rows, int32_t channels,
                        int32_t out, int32_t dtype, void* y, void* ws, size_t ws_bytes, void* stream)
{
    using namespace gs;
    if (!four_sizes_ok(rows, channels) || out < 1 || out > (1 << 17) || !dtype_ok(dtype)) return GS_ERR_INVALID_ARGUMENT;
    if (rows == 0) return GS_OK;
    if (!x || !x->data || !codes || !codes->data || !scales || !scales->data || !y) return GS_ERR_INVALID_ARGUMENT;
    const size_t need = gs_linear_fp4_workspace_bytes(rows, channels, out);
    if (need && (!ws || ((uintptr_t)ws & 15) || ws_bytes < need)) return GS_ERR_INVALID_ARGUMENT;
    if (!four_rows_ok(x, channels, elem_bytes(dtype), 16) || !four_rows_ok(codes, channels / 2, 1, 16) || !four_rows_ok(scales, scale_bytes_of(channels), 1, 4) ||
        (uintptr_t)y % elem_bytes(dtype) || ((rows + 63) / 64) * ((out + 63) / 64) >= (1 << 23))
        return GS_ERR_UNSUPPORTED;
    const hipStream_t s = (hipStream_t)stream;
    FourArgs p{};
    p.b = {{(const char*)codes->data, (const char*)scales->data}, {codes->stride, scales->stride}, out};
    p.walk = {channels / 4, (channels + 127) / 128, 0, (channels + 127) / 128};
    p.y = y;
    p.m = rows;
    p.n = out;
    if (rows <= FOUR_FEW) {
        const hipError_t e = dtype == GS_F32   ? few_as<float>(p, x, s)
                             : dtype == GS_F16 ? few_as<f16>(p, x, s)
                                               : few_as<bf16>(p, x, s);
        return e == hipSuccess ? GS_OK : GS_ERR_HIP;
    }
    char* xc = (char*)ws;
    char* xs = xc + ((size_t)rows * (channels / 2) + 15) / 16 * 16;
    if (quantise_as(dtype, x, xc, xs, rows, channels, s) != hipSuccess) return GS_ERR_HIP;
    p.a = {{xc, xs}, {channels / 2, scale_bytes_of(channels)}, rows};
    const hipError_t e = dtype == GS_F32 ? product_as<float>(p, s) : (dtype == GS_F16 ? product_as<f16>(p, s) : product_as<bf16>(p, s));
    return e == hipSuccess ? GS_OK : GS_ERR_HIP;
}

}  // extern "C"
