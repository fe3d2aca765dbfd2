// gs_layer_norm_fwd and gs_layer_norm_bwd: layer norm over the channels of
// each row, and its gradients.
//
// Each element is read and written once in either direction, so both are bound
// by HBM: 32640 x 2048 bf16 forward 59 us (4.5 TB/s), back 84 (4.8 TB/s) and 6
// for the sums. NT threads hold a row in registers; a workgroup walks over a
// contiguous run of rows with the weights of its columns in registers, and the
// next row is loaded (as it lies in memory, 4 registers for 16 bytes) before
// the present one's reductions, so that its latency runs behind them.
//
// The mean is subtracted before the squares are summed (two reductions a row in
// the forward pass): the sum of squares minus the squared mean would cancel
// where a row is far off zero. What the differences still sum to, the roundings
// of the mean, is summed beside their squares and taken off too. The backward pass needs mean d and mean d xh of
// one reduction. The sums over rows are kept per column along the run,
// written once per run, and added in a fixed order by k_layer_sums.
//
// All of it is fp32 between the loads and the stores, with one rounding per
// result.
#include "norm.h"

namespace gs {

// The columns a thread holds, as Cols, but for any channel count and alignment:
// pack i covers [(i NT + t) VEC, + VEC), n[i] of them below the channel count.
// Whole packs are loaded at once wherever they start (a vector access needs its
// element's alignment only), the last one of a ragged row element by element.
template <int VEC, int NV, int NT>
struct RaggedCols {
    int base, n[NV];
    __device__ __forceinline__ RaggedCols(int t, int channels) : base(t * VEC)
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) n[i] = min(max(channels - at(i), 0), VEC);
    }
    __device__ __forceinline__ int at(int i) const { return base + i * NT * VEC; }
    __device__ __forceinline__ bool has(int i, int e) const { return e < n[i]; }
    template <typename T>
    struct Raw {
        T v[NV][VEC];
    };
    template <typename T, int N>
    struct Unaligned {
        T v[N];
    } __attribute__((packed, aligned(sizeof(T))));
    template <typename T, int N>
    static __device__ __forceinline__ void copy(T* to, const T* from)
    {
        *(Unaligned<T, N>*)to = *(const Unaligned<T, N>*)from;
    }
    template <typename T>
    __device__ __forceinline__ void load(const T* p, Raw<T>& out) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (n[i] == VEC) {
                copy<T, VEC>(out.v[i], p + at(i));
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) out.v[i][e] = has(i, e) ? p[at(i) + e] : (T)0.f;
            }
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* p, const float (&in)[NV][VEC]) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            T v[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[e] = (T)in[i][e];
            if (n[i] == VEC) {
                copy<T, VEC>(p + at(i), v);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (has(i, e)) p[at(i) + e] = v[e];
            }
        }
    }
    // fp32 vectors of the channels, or `other` where there is none
    __device__ __forceinline__ void load_vec(const float* p, float (&out)[NV][VEC], float other) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (p && n[i] == VEC) {
#pragma unroll
                for (int e = 0; e < VEC; e += 4) copy<float, 4>(out[i] + e, p + at(i) + e);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) out[i][e] = p && has(i, e) ? p[at(i) + e] : other;
            }
        }
    }
};

struct LayerArgs {
    const void *x, *gy;
    const float *w, *b;
    void* out;                 // y or gx
    float* stats;              // [2][rows]: mean, 1 / deviation
    float* part;               // backward: [runs][2][channels], sums of gy xh and gy
    int64_t rows, run, stride_x, stride_gy;
    int32_t channels;
    float eps;
};

// 1 / sqrt(v), one rounding off at most; the hardware's takes no subnormals.
__device__ __forceinline__ float inverse_root(float v)
{
    const bool tiny = v < 0x1p-100f;
    return __builtin_amdgcn_rsqf(tiny ? v * 0x1p60f : v) * (tiny ? 0x1p30f : 1.f);
}

// FULL: the threads hold exactly a row; else what is past it is masked.
template <typename T, int VEC, int NV, int NT, int AHEAD, bool FULL>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_layer_fwd(const LayerArgs a)
{
    constexpr int PER = NT < 256 ? 256 / NT : 1;
    __shared__ float s_buf[NT > 64 ? 2 * (NT / 64) : 1], s_buf2[NT > 64 ? 2 * (NT / 64) * 2 : 1];
    using C = RaggedCols<VEC, NV, NT>;
    const C col(threadIdx.x % NT, a.channels);
    const int64_t run = (int64_t)blockIdx.x * PER + threadIdx.x / NT;
    const int64_t r0 = run * a.run, r1 = r0 + a.run < a.rows ? r0 + a.run : a.rows;
    if (r0 >= a.rows) return;  // whole waves (NT >= 64); with NT > 64 the whole workgroup
    const T* px = (const T*)a.x;
    const float inv = 1.f / (float)a.channels;
    typename C::template Raw<T> next[AHEAD];
#pragma unroll
    for (int d = 0; d < AHEAD; ++d)
        if (r0 + d < r1) col.load(px + (r0 + d) * a.stride_x, next[d]);
    float w[NV][VEC], b[NV][VEC], mask[NV][VEC];
    col.load_vec(a.w, w, 1.f);
    col.load_vec(a.b, b, 0.f);
    GS_EACH(mask[i][e] = col.has(i, e) ? 1.f : 0.f)
    int flip = 0;
    const auto one = [&](int64_t r, typename C::template Raw<T>& raw) __attribute__((always_inline)) {
        float x[NV][VEC], sum[1] = {0.f};
        GS_EACH(x[i][e] = (float)raw.v[i][e]; sum[0] += x[i][e])
        if (r + AHEAD < r1) col.load(px + (r + AHEAD) * a.stride_x, raw);
        row_sums<NT, 1>(sum, s_buf, flip);
        flip ^= 1;
        const float mean = sum[0] * inv;
        float v[2] = {0.f, 0.f};
        GS_EACH(x[i][e] -= mean; const float d = FULL ? x[i][e] : x[i][e] * mask[i][e]; v[0] += d; v[1] = fmaf(d, d, v[1]))
        row_sums<NT, 2>(v, s_buf2, flip);
        const float rest = v[0] * inv, var = fmaf(-rest, rest, v[1] * inv);
        const float rs = inverse_root((var < 0.f ? 0.f : var) + a.eps);
        const float shift = -rest * rs;
        GS_EACH(x[i][e] = fmaf(fmaf(x[i][e], rs, shift), w[i][e], b[i][e]))
        col.store((T*)a.out + r * a.channels, x);
        if (threadIdx.x % NT == 0) {
            a.stats[r] = mean + rest;
            a.stats[a.rows + r] = rs;
        }
    };
    for (int64_t r = r0; r < r1; r += AHEAD)
#pragma unroll
        for (int d = 0; d < AHEAD; ++d)
            if (r + d < r1) one(r + d, next[d]);
}

template <typename T, int VEC, int NV, int NT, int AHEAD, bool FULL>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_layer_bwd(const LayerArgs a)
{
    constexpr int PER = NT < 256 ? 256 / NT : 1;
    __shared__ float s_buf[NT > 64 ? 2 * (NT / 64) * 2 : 1];
    using C = RaggedCols<VEC, NV, NT>;
    const C col(threadIdx.x % NT, a.channels);
    const int64_t run = (int64_t)blockIdx.x * PER + threadIdx.x / NT;
    const int64_t r0 = run * a.run, r1 = r0 + a.run < a.rows ? r0 + a.run : a.rows;
    if (r0 >= a.rows) return;  // whole waves (NT >= 64); with NT > 64 the whole workgroup
    const T *px = (const T*)a.x, *pg = (const T*)a.gy;
    const float inv = 1.f / (float)a.channels;
    typename C::template Raw<T> next_x[AHEAD], next_g[AHEAD];
#pragma unroll
    for (int d = 0; d < AHEAD; ++d)
        if (r0 + d < r1) {
            col.load(px + (r0 + d) * a.stride_x, next_x[d]);
            col.load(pg + (r0 + d) * a.stride_gy, next_g[d]);
        }
    float w[NV][VEC], sum_w[NV][VEC], sum_b[NV][VEC];
    col.load_vec(a.w, w, 1.f);
    GS_EACH(sum_w[i][e] = 0.f; sum_b[i][e] = 0.f)
    int flip = 0;
    const auto one = [&](int64_t r, typename C::template Raw<T>& raw_x, typename C::template Raw<T>& raw_g) __attribute__((always_inline)) {
        const float mean = a.stats[r], rs = a.stats[a.rows + r];
        float xh[NV][VEC], d[NV][VEC], v[2] = {0.f, 0.f};
        // past the channels gy is zero, and with it every term (of x there, mean times rs may pass fp32)
        GS_EACH(xh[i][e] = FULL || col.has(i, e) ? ((float)raw_x.v[i][e] - mean) * rs : 0.f; const float g = (float)raw_g.v[i][e];
                sum_w[i][e] = fmaf(g, xh[i][e], sum_w[i][e]); sum_b[i][e] += g; d[i][e] = g * w[i][e];
                v[0] += d[i][e]; v[1] = fmaf(d[i][e], xh[i][e], v[1]))
        if (r + AHEAD < r1) {
            col.load(px + (r + AHEAD) * a.stride_x, raw_x);
            col.load(pg + (r + AHEAD) * a.stride_gy, raw_g);
        }
        row_sums<NT, 2>(v, s_buf, flip);
        flip ^= 1;
        const float m0 = v[0] * inv, m1 = v[1] * inv;
        GS_EACH(d[i][e] = rs * fmaf(-m1, xh[i][e], d[i][e] - m0))
        col.store((T*)a.out + r * a.channels, d);
    };
    for (int64_t r = r0; r < r1; r += AHEAD)
#pragma unroll
        for (int d = 0; d < AHEAD; ++d)
            if (r + d < r1) one(r + d, next_x[d], next_g[d]);
    if (a.part) {
        float* p = a.part + run * 2 * a.channels;
        col.store(p, sum_w);
        col.store(p + a.channels, sum_b);
    }
}

// gw (blockIdx.y 0) and gb (1) from the runs' sums.
__global__ __launch_bounds__(SUMS_COLS* SUMS_SLICES) void k_layer_sums(const float* __restrict__ part,
                                                                       float* __restrict__ gw, float* __restrict__ gb,
                                                                       int64_t runs, int32_t channels)
{
    __shared__ float s_buf[SUMS_SLICES][SUMS_COLS];
    const int c = blockIdx.x * SUMS_COLS + threadIdx.x % SUMS_COLS;
    float* out = blockIdx.y ? gb : gw;
    if (!out) return;
    const float t = slice_sum(part + (blockIdx.y ? channels : 0), 0, runs, 2 * (int64_t)channels, c, c < channels, s_buf);
    if (c < channels && threadIdx.x < SUMS_COLS) out[c] = t;
}

template <typename T, int VEC, int NV, int NT>
static hipError_t layer_launch(const LayerArgs& a, bool backward, hipStream_t s)
{
    constexpr int PER = NT < 256 ? 256 / NT : 1, THREADS = NT < 256 ? 256 : NT;
    constexpr int AHEAD = 2, BACK = 1;  // rows loaded ahead; 3 and 4 took no less
    const dim3 grid(grid_for((uint64_t)((a.rows + a.run - 1) / a.run), PER));
    const bool full = a.channels == VEC * NV * NT;
    if (backward && full)
        hipLaunchKernelGGL((k_layer_bwd<T, VEC, NV, NT, BACK, true>), grid, dim3(THREADS), 0, s, a);
    else if (backward)
        hipLaunchKernelGGL((k_layer_bwd<T, VEC, NV, NT, BACK, false>), grid, dim3(THREADS), 0, s, a);
    else if (full)
        hipLaunchKernelGGL((k_layer_fwd<T, VEC, NV, NT, AHEAD, true>), grid, dim3(THREADS), 0, s, a);
    else
        hipLaunchKernelGGL((k_layer_fwd<T, VEC, NV, NT, AHEAD, false>), grid, dim3(THREADS), 0, s, a);
    return hipGetLastError();
}

// The fewest threads that hold a row in registers: one wave up to 16 values a
// thread (no barrier per row), then 256 threads, then 1024. For 2048 columns of
// bf16 one wave, with 32 values a thread, took 104 us forward and 197 back, 256
// threads 60 and 87.
template <typename T, int VEC>
static hipError_t layer_by_width(const LayerArgs& a, bool backward, hipStream_t s)
{
    const int64_t packs = (a.channels + VEC - 1) / VEC;
    if (packs <= 64) return layer_launch<T, VEC, 1, 64>(a, backward, s);
    if (packs <= 128) return layer_launch<T, VEC, 2, 64>(a, backward, s);
    if (packs <= 256) return layer_launch<T, VEC, 1, 256>(a, backward, s);
    if (packs <= 512) return layer_launch<T, VEC, 2, 256>(a, backward, s);
    if (packs <= 1024) return layer_launch<T, VEC, 1, 1024>(a, backward, s);
    if (packs <= 2048) return layer_launch<T, VEC, 2, 1024>(a, backward, s);
    return layer_launch<T, VEC, 4, 1024>(a, backward, s);
}

static hipError_t layer_dispatch(const LayerArgs& a, int32_t dtype, bool backward, hipStream_t s)
{
    switch (dtype) {
        case GS_F32: return layer_by_width<float, 4>(a, backward, s);
        case GS_F16: return layer_by_width<f16, 8>(a, backward, s);
        default: return layer_by_width<bf16, 8>(a, backward, s);
    }
}

static bool layer_sizes_ok(int64_t rows, int32_t channels)
{
    return rows >= 0 && rows <= ((int64_t)1 << 40) && channels >= 1 && channels <= 16384;
}

// Rows of an input: aligned to the element, and their strides so small that no
// offset in bytes passes 63 bits.
static bool layer_rows_ok(const gs_matrix* m, int32_t dtype)
{
    return m && m->data && ((uintptr_t)m->data % elem_bytes(dtype)) == 0 && m->stride >= 0 && m->stride < ((int64_t)1 << 20);
}

}  // namespace gs

extern "C" {

gs_status gs_layer_norm_fwd(const gs_matrix* x, const float* w, const float* b, void* y, float* stats, int64_t rows,
                            int32_t channels, float eps, int32_t dtype, void* stream)
{
    using namespace gs;
    if (!layer_sizes_ok(rows, channels) || !dtype_ok(dtype) || !(eps >= 0.f)) return GS_ERR_INVALID_ARGUMENT;
    if (rows == 0) return GS_OK;
    if (!layer_rows_ok(x, dtype) || !y || !stats) return GS_ERR_INVALID_ARGUMENT;
    LayerArgs a{};
    a.x = x->data;
    a.stride_x = x->stride;
    a.w = w;
    a.b = b;
    a.out = y;
    a.stats = stats;
    a.rows = rows;
    a.channels = channels;
    a.eps = eps;
    a.run = run_rows(rows, FWD_RUNS);
    return layer_dispatch(a, dtype, false, (hipStream_t)stream) == hipSuccess ? GS_OK : GS_ERR_HIP;
}

size_t gs_layer_norm_bwd_workspace_bytes(int64_t rows, int32_t channels)
{
    using namespace gs;
    if (!layer_sizes_ok(rows, channels)) return 0;
    const int64_t run = run_rows(rows, BWD_RUNS), runs = (rows + run - 1) / run;
    return (size_t)runs * 2 * (size_t)channels * 4 + 64;
}

gs_status gs_layer_norm_bwd(const gs_matrix* gy, const gs_matrix* x, const float* w, const float* stats, void* gx,
                            float* gw, float* gb, int64_t rows, int32_t channels, int32_t dtype, void* ws,
                            size_t ws_bytes, void* stream)
{
    using namespace gs;
    if (!layer_sizes_ok(rows, channels) || !dtype_ok(dtype)) return GS_ERR_INVALID_ARGUMENT;
    if (!ws || ((uintptr_t)ws & 15) || ws_bytes < gs_layer_norm_bwd_workspace_bytes(rows, channels))
        return GS_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (!layer_rows_ok(gy, dtype) || !layer_rows_ok(x, dtype) || !stats || !gx)) return GS_ERR_INVALID_ARGUMENT;
    const hipStream_t s = (hipStream_t)stream;
    LayerArgs a{};
    a.run = run_rows(rows, BWD_RUNS);
    const int64_t runs = (rows + a.run - 1) / a.run;
    if (rows > 0) {
        a.x = x->data;
        a.stride_x = x->stride;
        a.gy = gy->data;
        a.stride_gy = gy->stride;
        a.w = w;
        a.out = gx;
        a.stats = (float*)stats;
        a.part = gw || gb ? (float*)ws : nullptr;
        a.rows = rows;
        a.channels = channels;
        if (layer_dispatch(a, dtype, true, s) != hipSuccess) return GS_ERR_HIP;
    }
    if (gw || gb) {  // zeros when there are no rows
        hipLaunchKernelGGL(k_layer_sums, dim3(grid_for((uint64_t)channels, SUMS_COLS), 2), dim3(SUMS_COLS * SUMS_SLICES), 0, s,
                           (const float*)ws, gw, gb, runs, channels);
        GS_CHECK_LAUNCH();
    }
    return GS_OK;
}

}  // extern "C"
