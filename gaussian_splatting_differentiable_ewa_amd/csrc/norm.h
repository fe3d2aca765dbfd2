// Shared by the norms (norm_gate.hip, layer_norm.hip): rows held in registers,
// their reductions, and sums over runs of rows.
#pragma once

#include "tokens.h"

namespace gs {

// A barrier for LDS alone: __syncthreads also waits for the loads of the next
// row and the stores of the last one.
__device__ __forceinline__ void lds_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

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
        lds_barrier();
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

#define GS_EACH(body)                        \
    _Pragma("unroll") for (int i = 0; i < NV; ++i) { \
        _Pragma("unroll") for (int e = 0; e < VEC; ++e) { body; } \
    }

// Sums over runs, 32 columns by 32 slices of the runs a workgroup, each slice
// in order and the slices in order.
constexpr int SUMS_COLS = 32, SUMS_SLICES = 32;

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

// Rows per run: enough runs to fill the 256 CUs several times over. The
// backward writes 1 or 2 fp32 rows of sums per run, so it takes fewer (512 or
// 768 of them leave CUs idle at the end and are slower than 1024).
static int64_t run_rows(int64_t rows, int64_t want) { return std::max<int64_t>(1, (rows + want - 1) / want); }

constexpr int64_t FWD_RUNS = 4096, BWD_RUNS = 1024;

}  // namespace gs
