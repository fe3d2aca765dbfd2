// Device-side helpers shared by the token operators (rope.hip, norm_gate.hip,
// block_select.hip, block_attn.hip, block_attn_bwd.hip): element types,
// vector loads and the token views.
#pragma once

#include "internal.h"

namespace gs {

typedef __bf16 bf16;
typedef _Float16 f16;

// A token tensor [batch][tokens][heads][dim] as the kernels see it.
template <typename T>
struct View {
    T* data;
    int64_t sb, st, sh;
    __device__ __forceinline__ T* at(int64_t b, int64_t t, int64_t h) const { return data + b * sb + t * st + h * sh; }
};

template <typename T>
inline View<T> view_of(const gs_tokens* t)
{
    if (!t) return {nullptr, 0, 0, 0};
    return {(T*)t->data, t->stride_b, t->stride_t, t->stride_h};
}

// N consecutive elements as one load or store of up to 16 bytes.
template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
    T v[N];
};

template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* p, float (&out)[N])
{
    const Pack<T, N> x = *(const Pack<T, N>*)p;
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = (float)x.v[i];
}

template <typename T, int N>
__device__ __forceinline__ void store_f32(T* p, const float (&in)[N])
{
    Pack<T, N> x;
#pragma unroll
    for (int i = 0; i < N; ++i) x.v[i] = (T)in[i];
    *(Pack<T, N>*)p = x;
}

inline int elem_bytes(int32_t dtype) { return dtype == GS_F32 ? 4 : 2; }

inline bool dtype_ok(int32_t dtype) { return dtype == GS_F32 || dtype == GS_F16 || dtype == GS_BF16; }

// Whether every row [dim] of the view starts on a multiple of `bytes`
// (strides of dimensions of size 1 are never used).
inline bool rows_aligned(const gs_tokens* t, int64_t batch, int64_t tokens, int64_t heads, int elem, int bytes)
{
    const int64_t per = bytes / elem;
    return ((uintptr_t)t->data % bytes) == 0 && (batch <= 1 || t->stride_b % per == 0) &&
           (tokens <= 1 || t->stride_t % per == 0) && (heads <= 1 || t->stride_h % per == 0);
}

}  // namespace gs
