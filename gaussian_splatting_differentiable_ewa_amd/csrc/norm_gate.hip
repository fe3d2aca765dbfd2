// gs_norm_gate_fwd and gs_norm_gate_bwd: the norm after a block with its gate
// and residual scale, and the norm before the next one.
//
// Both directions read and write each element once and are bound by HBM. NT
// threads hold one row in registers; a workgroup walks over a contiguous run
// of rows with the weights and the gate of its columns in registers, so the
// fp32 vectors (3 x 4 bytes per channel) are read once per run instead of
// once per row, which would be more bytes than the row itself.
//
// The backward pass needs two means per row, the second of them of a quantity
// that contains the first. With t = gy + r1 (d1 - yh m1), u = scale gate w2 fh:
//   sum d2 fh = sum u t = sum u (gy + r1 d1) - r1 m1 sum u yh,
// so both come from three sums of one reduction. The sums over rows (weights
// and gates) are kept per column in registers along the run, written once
// per run and gate, and added in a fixed order by k_norm_sums.
//
// All of it is fp32 between the loads and the stores, with one rounding per
// result: h comes from the unrounded y.
//
// Measured, 32640 rows of 2048 bf16 channels: forward 97.5 us (4 tensors, 5.5
// TB/s), backward 178 us (6 tensors, 4.5 TB/s; one row's loads wait behind the
// last one's reduction, and loading a row ahead needs registers that cost as
// much occupancy as it gains), sums 15 us. 7200 rows of 1027 fp32 channels
// (rows off 16 bytes, so 4 bytes an access): 21, 34 and 10 us, 5.6 and 5.2
// TB/s (it fits the last-level cache).
#include "tokens.h"

namespace gs {

// Sums of N values over the NT threads that share a row. `buf` holds 2 x
// (NT / 64) x N floats and alternates by `flip`, so one barrier per call is
// enough: a wave can be at most one call ahead of the slowest.
template <int NT, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* buf, int flip)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
    if constexpr (NT > 64) {
        constexpr int W = NT / 64;
        float* mine = buf + flip * W * N;
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) mine[wave * N + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) s += mine[w * N + i];
            v[i] = s;
        }
    }
}

// The columns a thread holds: pack i covers [(i NT + t) VEC, + VEC), all of
// it below the channel count or none of it.
template <int VEC, int NV, int NT>
struct Cols {
    int base;
    bool on[NV];
    __device__ __forceinline__ Cols(int t, int channels) : base(t * VEC)
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) on[i] = base + i * NT * VEC < channels;
    }
    __device__ __forceinline__ int at(int i) const { return base + i * NT * VEC; }
    template <typename T>
    __device__ __forceinline__ void load(const T* p, float (&out)[NV][VEC], float other = 0.f) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (on[i] && p) {
                load_f32<T, VEC>(p + at(i), out[i]);
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) out[i][e] = other;
            }
        }
    }
    // fp32 vectors of the channels: 16 bytes at a time where VEC allows
    __device__ __forceinline__ void load_vec(const float* p, float (&out)[NV][VEC], float other) const
    {
        constexpr int Q = VEC >= 4 ? 4 : VEC;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < VEC; e += Q) {
                float x[Q];
#pragma unroll
                for (int j = 0; j < Q; ++j) x[j] = other;
                if (on[i] && p) load_f32<float, Q>(p + at(i) + e, x);
#pragma unroll
                for (int j = 0; j < Q; ++j) out[i][e + j] = x[j];
            }
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* p, const float (&in)[NV][VEC]) const
    {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (on[i]) store_f32<T, VEC>(p + at(i), in[i]);
    }
    __device__ __forceinline__ void store_vec(float* p, const float (&in)[NV][VEC]) const
    {
        constexpr int Q = VEC >= 4 ? 4 : VEC;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!on[i]) continue;
#pragma unroll
            for (int e = 0; e < VEC; e += Q) {
                float x[Q];
#pragma unroll
                for (int j = 0; j < Q; ++j) x[j] = in[i][e + j];
                store_f32<float, Q>(p + at(i) + e, x);
            }
        }
    }
};

struct NormArgs {
    const void *x, *f, *gy, *gh;
    const float *gate, *w_post, *w_pre;
    void *o0, *o1;      // forward: y, h; backward: gx, gf
    float* stats;
    float *part_a, *part_w;  // backward: per (run, gate) and per run sums
    int64_t rows, per_gate, run;
    int32_t channels;
    float scale, eps;
};

#define GS_EACH(body)                        \
    _Pragma("unroll") for (int i = 0; i < NV; ++i) { \
        _Pragma("unroll") for (int e = 0; e < VEC; ++e) { body; } \
    }

// One run of rows per NT threads (256 / NT runs per workgroup when NT < 256).
template <typename T, int VEC, int NV, int NT>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_norm_fwd(const NormArgs a)
{
    constexpr int PER = NT < 256 ? 256 / NT : 1;
    __shared__ float s_buf[NT > 64 ? 2 * (NT / 64) : 1];
    const Cols<VEC, NV, NT> col(threadIdx.x % NT, a.channels);
    const int64_t run = (int64_t)blockIdx.x * PER + threadIdx.x / NT;
    const int64_t r0 = run * a.run, r1 = r0 + a.run < a.rows ? r0 + a.run : a.rows;
    const T* px = (const T*)a.x;
    const T* pf = (const T*)a.f;
    const float inv = 1.f / (float)a.channels;
    float w2[NV][VEC], w1[NV][VEC], g[NV][VEC];
    col.load_vec(pf ? a.w_post : nullptr, w2, 1.f);
    col.load_vec(a.w_pre, w1, 1.f);
    int64_t seg = -1;
    int flip = 0;
    for (int64_t r = r0; r < r1; ++r) {
        float x[NV][VEC], f[NV][VEC];
        col.load(px + r * a.channels, x);
        float r2 = 0.f;
        if (pf) {
            col.load(pf + r * a.channels, f);
            const int64_t s = r / a.per_gate;
            if (s != seg) {
                seg = s;
                col.load_vec(a.gate ? a.gate + s * a.channels : nullptr, g, 1.f);
                GS_EACH(g[i][e] *= a.scale * w2[i][e])
            }
            float sum[1] = {0.f};
            GS_EACH(sum[0] = fmaf(f[i][e], f[i][e], sum[0]))
            row_sums<NT, 1>(sum, s_buf, flip);
            flip ^= 1;
            r2 = 1.f / sqrtf(fmaf(sum[0], inv, a.eps));
            GS_EACH(x[i][e] = fmaf(g[i][e], f[i][e] * r2, x[i][e]))
            col.store((T*)a.o0 + r * a.channels, x);
        }
        float sum[1] = {0.f};
        GS_EACH(sum[0] = fmaf(x[i][e], x[i][e], sum[0]))
        row_sums<NT, 1>(sum, s_buf, flip);
        flip ^= 1;
        const float rp = 1.f / sqrtf(fmaf(sum[0], inv, a.eps));
        GS_EACH(x[i][e] = x[i][e] * rp * w1[i][e])
        col.store((T*)a.o1 + r * a.channels, x);
        if (threadIdx.x % NT == 0) {
            a.stats[r] = r2;
            a.stats[a.rows + r] = rp;
        }
    }
}

template <typename T, int VEC, int NV, int NT>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_norm_bwd(const NormArgs a)
{
    constexpr int PER = NT < 256 ? 256 / NT : 1;
    __shared__ float s_buf[NT > 64 ? 2 * (NT / 64) * 3 : 1];
    const Cols<VEC, NV, NT> col(threadIdx.x % NT, a.channels);
    const int64_t run = (int64_t)blockIdx.x * PER + threadIdx.x / NT;
    const int64_t r0 = run * a.run, r1 = r0 + a.run < a.rows ? r0 + a.run : a.rows;
    if (r0 >= a.rows) return;  // whole waves (NT >= 64); with NT > 64 the whole workgroup
    const T *px = (const T*)a.x, *pf = (const T*)a.f, *pgy = (const T*)a.gy, *pgh = (const T*)a.gh;
    const float inv = 1.f / (float)a.channels;
    float w1[NV][VEC], g[NV][VEC], sum_w[NV][VEC], sum_a[NV][VEC];
    col.load_vec(a.w_pre, w1, 1.f);
    GS_EACH(sum_w[i][e] = 0.f; sum_a[i][e] = 0.f; g[i][e] = 0.f)
    int64_t seg = -1;
    int flip = 0;
    for (int64_t r = r0; r < r1; ++r) {
        const int64_t o = r * a.channels;
        float x[NV][VEC], f[NV][VEC], gy[NV][VEC], gh[NV][VEC];
        col.load(px + o, x);
        col.load(pf ? pf + o : nullptr, f);
        col.load(pgy ? pgy + o : nullptr, gy);
        col.load(pgh + o, gh);
        const float rp = a.stats[a.rows + r];
        float r2 = 0.f;
        if (pf) {
            r2 = a.stats[r];
            const int64_t s = r / a.per_gate;
            if (s != seg) {
                if (seg >= 0) {
                    col.store_vec(a.part_a + (run + seg) * a.channels, sum_a);
                    GS_EACH(sum_a[i][e] = 0.f)
                }
                seg = s;
                float w2[NV][VEC];
                col.load_vec(a.gate ? a.gate + s * a.channels : nullptr, g, 1.f);
                col.load_vec(a.w_post, w2, 1.f);
                GS_EACH(g[i][e] *= a.scale * w2[i][e])
            }
        }
        float v[3] = {0.f, 0.f, 0.f};
        GS_EACH(f[i][e] *= r2; x[i][e] = fmaf(g[i][e], f[i][e], x[i][e]) * rp;
                const float d1 = gh[i][e] * w1[i][e]; sum_w[i][e] = fmaf(gh[i][e], x[i][e], sum_w[i][e]);
                gy[i][e] = fmaf(rp, d1, gy[i][e]); const float u = g[i][e] * f[i][e];
                v[0] = fmaf(d1, x[i][e], v[0]); v[1] = fmaf(u, gy[i][e], v[1]); v[2] = fmaf(u, x[i][e], v[2]))
        row_sums<NT, 3>(v, s_buf, flip);
        flip ^= 1;
        const float m1 = rp * v[0] * inv;
        const float m2 = (v[1] - m1 * v[2]) * inv;
        GS_EACH(gy[i][e] = fmaf(-m1, x[i][e], gy[i][e]))
        col.store((T*)a.o0 + o, gy);
        if (pf) {
            GS_EACH(sum_a[i][e] = fmaf(gy[i][e], f[i][e], sum_a[i][e]);
                    f[i][e] = r2 * fmaf(-m2, f[i][e], gy[i][e] * g[i][e]))
            col.store((T*)a.o1 + o, f);
        }
    }
    col.store_vec(a.part_w + run * a.channels, sum_w);
    if (pf) col.store_vec(a.part_a + (run + seg) * a.channels, sum_a);
}

// Sums over runs, 32 columns by 32 slices of the runs a workgroup, each slice
// in order and the slices in order. The workgroups of gate s: A[s] from the
// slots s + (runs that hold rows of s), times scale; then those of gw_pre;
// then, with few gates, those of gw_post, which add the gates' sums again
// instead of waiting for them in a launch of their own.
constexpr int SUMS_COLS = 32, SUMS_SLICES = 32, SUMS_GATES = 64;

__device__ __forceinline__ float slice_sum(const float* __restrict__ p, int64_t first, int64_t count, int64_t stride, int c,
                                           bool on, float (*s_buf)[SUMS_COLS])
{
    const int slice = threadIdx.x / SUMS_COLS, col = threadIdx.x % SUMS_COLS;
    float s = 0.f;
    if (on) {
        const int64_t per = (count + SUMS_SLICES - 1) / SUMS_SLICES;
        const int64_t lo = slice * per, hi = lo + per < count ? lo + per : count;
#pragma unroll 8
        for (int64_t k = lo; k < hi; ++k) s += p[(first + k) * stride + c];
    }
    s_buf[slice][col] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int k = 0; k < SUMS_SLICES; ++k) s += s_buf[k][col];
    __syncthreads();
    return s;
}

__global__ __launch_bounds__(SUMS_COLS* SUMS_SLICES) void k_norm_sums(
    const float* __restrict__ part_a, const float* __restrict__ part_w, const float* __restrict__ gate,
    const float* __restrict__ w_post, float* __restrict__ a_of_gate, float* __restrict__ ggate, float* __restrict__ gw_pre,
    float* __restrict__ gw_post, int64_t rows, int64_t per_gate, int64_t gates, int64_t run, int64_t runs, int32_t channels,
    float scale)
{
    __shared__ float s_buf[SUMS_SLICES][SUMS_COLS];
    const int columns = (channels + SUMS_COLS - 1) / SUMS_COLS;
    const int c = blockIdx.x % columns * SUMS_COLS + threadIdx.x % SUMS_COLS;
    const bool on = c < channels, first = on && threadIdx.x < SUMS_COLS;
    const int64_t s = blockIdx.x / columns;
    if (s == gates) {
        const float t = slice_sum(part_w, 0, runs, channels, c, on, s_buf);
        if (first && gw_pre) gw_pre[c] = t;
        return;
    }
    const auto of_gate = [&](int64_t g) {
        const int64_t lo = g * per_gate, end = lo + per_gate < rows ? lo + per_gate : rows;
        const int64_t c0 = lo / run, c1 = (end - 1) / run;
        return scale * slice_sum(part_a, g + c0, c1 - c0 + 1, channels, c, on, s_buf);
    };
    if (s > gates) {
        float t = 0.f;
        for (int64_t g = 0; g < gates; ++g) {
            const float x = of_gate(g);
            if (on) t += gate ? gate[g * channels + c] * x : x;
        }
        if (first) gw_post[c] = t;
        return;
    }
    const float t = of_gate(s);
    if (first) {
        a_of_gate[s * channels + c] = t;
        if (ggate) ggate[s * channels + c] = w_post ? w_post[c] * t : t;
    }
}

// gw_post = sum over (many) gates of gate A.
__global__ __launch_bounds__(SUMS_COLS* SUMS_SLICES) void k_norm_gw_post(const float* __restrict__ a_of_gate,
                                                                         const float* __restrict__ gate, int64_t gates,
                                                                         int32_t channels, float* __restrict__ gw_post)
{
    __shared__ float s_buf[SUMS_SLICES][SUMS_COLS];
    const int col = threadIdx.x % SUMS_COLS, slice = threadIdx.x / SUMS_COLS, c = blockIdx.x * SUMS_COLS + col;
    float s = 0.f;
    if (c < channels) {
        const int64_t per = (gates + SUMS_SLICES - 1) / SUMS_SLICES;
        const int64_t lo = slice * per, hi = lo + per < gates ? lo + per : gates;
#pragma unroll 8
        for (int64_t k = lo; k < hi; ++k) {
            const float x = a_of_gate[k * channels + c];
            s += gate ? gate[k * channels + c] * x : x;
        }
    }
    s_buf[slice][col] = s;
    __syncthreads();
    if (threadIdx.x < SUMS_COLS && c < channels) {
        s = 0.f;
        for (int k = 0; k < SUMS_SLICES; ++k) s += s_buf[k][col];
        gw_post[c] = s;
    }
}

// Rows per run: enough runs to fill the 256 CUs several times over. The
// backward writes 1 or 2 fp32 rows of sums per run, so it takes fewer (512 or
// 768 of them leave CUs idle at the end and are slower than 1024).
static int64_t run_rows(int64_t rows, int64_t want) { return std::max<int64_t>(1, (rows + want - 1) / want); }

constexpr int64_t FWD_RUNS = 4096, BWD_RUNS = 1024;

template <typename T, int VEC, int NV, int NT>
static hipError_t norm_launch(NormArgs& a, bool backward, hipStream_t s)
{
    constexpr int PER = NT < 256 ? 256 / NT : 1, THREADS = NT < 256 ? 256 : NT;
    const int64_t runs = (a.rows + a.run - 1) / a.run;
    const dim3 grid(grid_for((uint64_t)runs, PER));
    if (backward)
        hipLaunchKernelGGL((k_norm_bwd<T, VEC, NV, NT>), grid, dim3(THREADS), 0, s, a);
    else
        hipLaunchKernelGGL((k_norm_fwd<T, VEC, NV, NT>), grid, dim3(THREADS), 0, s, a);
    return hipGetLastError();
}

// The fewest threads that hold a row in registers: one wave up to 16 values a
// thread (no barrier per row), then 256 threads, then 1024.
template <typename T, int VEC>
static hipError_t norm_by_width(NormArgs& a, bool backward, bool wide, hipStream_t s)
{
    if (wide) {
        const int64_t packs = a.channels / VEC;
        if (packs <= 64) return norm_launch<T, VEC, 1, 64>(a, backward, s);
        if (packs <= 128) return norm_launch<T, VEC, 2, 64>(a, backward, s);
        if (packs <= 256) return norm_launch<T, VEC, 1, 256>(a, backward, s);
        if (packs <= 512) return norm_launch<T, VEC, 2, 256>(a, backward, s);
        if (packs <= 1024) return norm_launch<T, VEC, 1, 1024>(a, backward, s);
        if (packs <= 2048) return norm_launch<T, VEC, 2, 1024>(a, backward, s);
        return norm_launch<T, VEC, 4, 1024>(a, backward, s);
    }
    const int64_t c = a.channels;
    if (c <= 256) return norm_launch<T, 1, 4, 64>(a, backward, s);
    if (c <= 1024) return norm_launch<T, 1, 4, 256>(a, backward, s);
    if (c <= 2048) return norm_launch<T, 1, 8, 256>(a, backward, s);
    if (c <= 4096) return norm_launch<T, 1, 4, 1024>(a, backward, s);
    return norm_launch<T, 1, 16, 1024>(a, backward, s);
}

static hipError_t norm_dispatch(NormArgs& a, int32_t dtype, bool backward, hipStream_t s)
{
    // 16-byte accesses need every row (and the fp32 vectors) on 16 bytes
    const int vec = 16 / elem_bytes(dtype);
    uintptr_t all = 0;
    for (const void* p : {a.x, a.f, a.gy, a.gh, (const void*)a.gate, (const void*)a.w_post, (const void*)a.w_pre,
                          (const void*)a.o0, (const void*)a.o1})
        all |= (uintptr_t)p;
    const bool wide = a.channels % vec == 0 && (all & 15) == 0;
    switch (dtype) {
        case GS_F32: return norm_by_width<float, 4>(a, backward, wide, s);
        case GS_F16: return norm_by_width<f16, 8>(a, backward, wide, s);
        default: return norm_by_width<bf16, 8>(a, backward, wide, s);
    }
}

static bool norm_sizes_ok(int64_t rows, int32_t channels, int64_t rows_per_gate)
{
    return rows >= 0 && rows <= ((int64_t)1 << 40) && channels >= 1 && channels <= 16384 && rows_per_gate >= 1;
}

static int64_t gates_of(int64_t rows, int64_t rows_per_gate) { return rows / rows_per_gate + (rows % rows_per_gate != 0); }

}  // namespace gs

extern "C" {

gs_status gs_norm_gate_fwd(const void* x, const void* f, const float* gate, const float* w_post, const float* w_pre,
                           void* y, void* h, float* stats, int64_t rows, int32_t channels, int64_t rows_per_gate,
                           float scale, float eps, int32_t dtype, void* stream)
{
    using namespace gs;
    if (!norm_sizes_ok(rows, channels, rows_per_gate) || !dtype_ok(dtype) || !(eps >= 0.f))
        return GS_ERR_INVALID_ARGUMENT;
    if (rows == 0) return GS_OK;
    if (!x || !h || !stats || (f && !y)) return GS_ERR_INVALID_ARGUMENT;
    NormArgs a{};
    a.x = x;
    a.f = f;
    a.gate = f ? gate : nullptr;
    a.w_post = f ? w_post : nullptr;
    a.w_pre = w_pre;
    a.o0 = f ? y : nullptr;
    a.o1 = h;
    a.stats = stats;
    a.rows = rows;
    a.per_gate = rows_per_gate;
    a.channels = channels;
    a.scale = scale;
    a.eps = eps;
    a.run = run_rows(rows, FWD_RUNS);
    return norm_dispatch(a, dtype, false, (hipStream_t)stream) == hipSuccess ? GS_OK : GS_ERR_HIP;
}

size_t gs_norm_gate_bwd_workspace_bytes(int64_t rows, int32_t channels, int64_t rows_per_gate)
{
    using namespace gs;
    if (!norm_sizes_ok(rows, channels, rows_per_gate)) return 0;
    const int64_t run = run_rows(rows, BWD_RUNS), runs = (rows + run - 1) / run, gates = gates_of(rows, rows_per_gate);
    // per run: gw_pre's sums; per (run, gate): A's; per gate: A
    return (size_t)(runs + (runs + gates) + gates) * (size_t)channels * 4 + 64;
}

gs_status gs_norm_gate_bwd(const void* gy, const void* gh, const void* x, const void* f, const float* gate,
                           const float* w_post, const float* w_pre, const float* stats, void* gx, void* gf,
                           float* ggate, float* gw_post, float* gw_pre, int64_t rows, int32_t channels,
                           int64_t rows_per_gate, float scale, int32_t dtype, void* ws, size_t ws_bytes, void* stream)
{
    using namespace gs;
    if (!norm_sizes_ok(rows, channels, rows_per_gate) || !dtype_ok(dtype)) return GS_ERR_INVALID_ARGUMENT;
    if (!ws || ((uintptr_t)ws & 15) || ws_bytes < gs_norm_gate_bwd_workspace_bytes(rows, channels, rows_per_gate))
        return GS_ERR_INVALID_ARGUMENT;
    if (rows > 0 && (!gh || !x || !stats || !gx || (f && !gf))) return GS_ERR_INVALID_ARGUMENT;
    const hipStream_t s = (hipStream_t)stream;
    NormArgs a{};
    a.x = x;
    a.f = f;
    a.gy = gy;
    a.gh = gh;
    a.gate = f ? gate : nullptr;
    a.w_post = f ? w_post : nullptr;
    a.w_pre = w_pre;
    a.o0 = gx;
    a.o1 = f ? gf : nullptr;
    a.stats = (float*)stats;
    a.rows = rows;
    a.per_gate = rows_per_gate;
    a.channels = channels;
    a.scale = scale;
    a.run = run_rows(rows, BWD_RUNS);
    const int64_t runs = (rows + a.run - 1) / a.run, gates = gates_of(rows, rows_per_gate);
    // the sums are stored 16 bytes at a time: pad each section's start
    a.part_w = (float*)ws;
    a.part_a = a.part_w + (runs * channels + 3) / 4 * 4;
    float* a_of_gate = a.part_a + ((runs + gates) * channels + 3) / 4 * 4;
    const unsigned columns = grid_for((uint64_t)channels, SUMS_COLS);
    // with f absent only gw_pre is summed (gates taken as 0)
    const int64_t g = f ? gates : 0;
    const bool with_post = f && gw_post && g > 0 && g <= SUMS_GATES;
    if ((g + 2) * columns > ((int64_t)1 << 21)) return GS_ERR_UNSUPPORTED;  // 1024 threads each, below 2^32 in all
    if (rows > 0 && norm_dispatch(a, dtype, true, s) != hipSuccess) return GS_ERR_HIP;
    hipLaunchKernelGGL(k_norm_sums, dim3((unsigned)(columns * (g + 1 + with_post))), dim3(SUMS_COLS * SUMS_SLICES), 0, s,
                       a.part_a, a.part_w, a.gate, a.w_post, a_of_gate, ggate, gw_pre, gw_post, rows, rows_per_gate, g, a.run,
                       runs, channels, scale);
    GS_CHECK_LAUNCH();
    // without rows f may be null because it is empty: its sum is zero, and written
    if ((f || rows == 0) && gw_post && !with_post) {
        hipLaunchKernelGGL(k_norm_gw_post, dim3(columns), dim3(SUMS_COLS * SUMS_SLICES), 0, s, a_of_gate, a.gate, gates,
                           channels, gw_post);
        GS_CHECK_LAUNCH();
    }
    return GS_OK;
}

}  // extern "C"
