// gs_rope_axes: rotary positions over (view, row, column) on queries and keys.
//
// Each element is read and written once, so the pass is bound by HBM. A
// thread owns VEC pairs (16 bytes of either half) of one token and walks over
// the heads of q and then k with them: the angle's sine and cosine, 8 of
// them, are formed once for ROPE_HEADS heads instead of once per element.
//
// Measured: 32640 tokens, 16 + 16 heads of dim 128, bf16: 100 us, 5.3 TB/s of
// reads and writes (the library's copy kernel: 5.1). 256 tokens, 8 + 8 heads of
// dim 64: 6 us, the latency of one wave (position, frequencies, sine, data).
#include "tokens.h"

namespace gs {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_HEADS = 4;  // heads a thread rotates with one set of sines

struct RopeArgs {
    int64_t batch, tokens, items, stride_pos_b;
    int32_t heads_q, heads_k, half, chunks, slices;
    int32_t p0, p1, p2;  // pairs of each axis
    int32_t interleaved, inverse;
};

// Sine and cosine of x f for any whole x of 32 bits. In fp32 the product alone
// would be off by up to half an ulp of itself, radians at far positions; so it
// is formed in fp64, with what fp64 rounds off, and reduced to +-pi by a 2 pi
// of two fp64 parts before it goes to fp32, again with its remainder e:
// cos(t + e) = cos t - e sin t, sin(t + e) = sin t + e cos t (e^2 < 2^-46).
__device__ __forceinline__ void turn_of(int32_t x, float f, float& sn, float& cs)
{
    constexpr double TWO_PI = 6.283185307179586477, TWO_PI_REST = 2.449293598294706e-16, PER = 0.15915494309189533577;
    const double xd = (double)x, fd = (double)f, t = xd * fd, k = rint(t * PER);
    double r = fma(-k, TWO_PI, t);
    r = fma(-k, TWO_PI_REST, r) + fma(xd, fd, -t);
    const float near = (float)r, e = (float)(r - (double)near);
    float s0, c0;
    sincosf(near, &s0, &c0);
    cs = fmaf(-e, s0, c0);
    sn = fmaf(e, c0, s0);
}

// VEC pairs at a time: contiguous elements of each half (or 2 VEC contiguous
// elements when interleaved). Sines and the rotation are fp32; each result is
// rounded once.
template <typename T, int VEC>
__global__ __launch_bounds__(ROPE_THREADS) void k_rope(View<const T> q, View<const T> k, View<T> qo, View<T> ko,
                                                       const int32_t* __restrict__ pos,
                                                       const float* __restrict__ freq, const RopeArgs a)
{
    const int64_t item = (int64_t)blockIdx.x * ROPE_THREADS + threadIdx.x;
    if (item >= a.items) return;
    const int64_t at = item / a.chunks;
    const int c = (int)(item - at * a.chunks);
    const int64_t token = at / a.slices;
    const int slice = (int)(at - token * a.slices);
    const int64_t b = token / a.tokens, l = token - b * a.tokens;
    const int32_t* p = pos + b * a.stride_pos_b + l * 3;
    const int32_t p0 = p[0], p1 = p[1], p2 = p[2];
    float cs[VEC], sn[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const int j = c * VEC + i;
        cs[i] = 1.f;
        sn[i] = 0.f;
        if (j < a.p0 + a.p1 + a.p2) {
            turn_of(j < a.p0 ? p0 : (j < a.p0 + a.p1 ? p1 : p2), freq[j], sn[i], cs[i]);
            if (a.inverse) sn[i] = -sn[i];
        }
    }
    const int o0 = a.interleaved ? 2 * c * VEC : c * VEC, o1 = a.interleaved ? o0 + VEC : o0 + a.half;
    for (int h = slice; h < a.heads_q + a.heads_k; h += a.slices) {
        const bool is_q = h < a.heads_q;
        const T* in = is_q ? q.at(b, l, h) : k.at(b, l, h - a.heads_q);
        T* out = is_q ? qo.at(b, l, h) : ko.at(b, l, h - a.heads_q);
        float u[VEC], w[VEC];
        load_f32<T, VEC>(in + o0, u);
        load_f32<T, VEC>(in + o1, w);
        if (a.interleaved) {
            float x[2 * VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) x[i] = u[i], x[VEC + i] = w[i];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float x0 = x[2 * i], x1 = x[2 * i + 1];
                x[2 * i] = fmaf(x0, cs[i], -(x1 * sn[i]));
                x[2 * i + 1] = fmaf(x0, sn[i], x1 * cs[i]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) u[i] = x[i], w[i] = x[VEC + i];
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float x0 = u[i], x1 = w[i];
                u[i] = fmaf(x0, cs[i], -(x1 * sn[i]));
                w[i] = fmaf(x0, sn[i], x1 * cs[i]);
            }
        }
        store_f32<T, VEC>(out + o0, u);
        store_f32<T, VEC>(out + o1, w);
    }
}

template <typename T, int VEC>
static gs_status rope_launch(const gs_tokens* q, const gs_tokens* k, const gs_tokens* qo, const gs_tokens* ko,
                             const int32_t* pos, const float* freq, RopeArgs a, hipStream_t stream)
{
    a.chunks = a.half / VEC;
    a.slices = (a.heads_q + a.heads_k + ROPE_HEADS - 1) / ROPE_HEADS;
    a.items = a.batch * a.tokens * a.slices * a.chunks;
    if (a.items > ((int64_t)1 << 31)) return GS_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((k_rope<T, VEC>), dim3(grid_for((uint64_t)a.items, ROPE_THREADS)), dim3(ROPE_THREADS), 0, stream,
                       view_of<const T>(q), view_of<const T>(k), view_of<T>(qo), view_of<T>(ko), pos, freq, a);
    GS_CHECK_LAUNCH();
    return GS_OK;
}

}  // namespace gs

extern "C" gs_status gs_rope_axes(const gs_tokens* q, const gs_tokens* k, const gs_tokens* q_out,
                                  const gs_tokens* k_out, int64_t batch, int64_t tokens, int32_t heads_q,
                                  int32_t heads_k, int32_t dim, int32_t dtype, const int32_t* pos,
                                  int64_t stride_pos_b, const float* freq, const int32_t* pairs, int32_t interleaved,
                                  int32_t inverse, void* stream)
{
    using namespace gs;
    if (!q || !q_out || !pairs || batch < 0 || tokens < 0 || heads_q < 0 || heads_k < 0 || dim < 2 || dim > 512 ||
        (dim & 1) || !dtype_ok(dtype) || (heads_k > 0 && (!k || !k_out)))
        return GS_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < 3; ++i)
        if (pairs[i] < 0 || pairs[i] > dim / 2) return GS_ERR_INVALID_ARGUMENT;
    if (pairs[0] + pairs[1] + pairs[2] > dim / 2) return GS_ERR_INVALID_ARGUMENT;
    // each factor first, so that the product cannot wrap
    const int64_t most = (int64_t)1 << 40, heads = (int64_t)heads_q + heads_k;
    if (batch > most || tokens > most || heads > (1 << 20)) return GS_ERR_INVALID_ARGUMENT;
    if (batch == 0 || tokens == 0 || heads == 0) return GS_OK;
    if (tokens > most / batch || heads * dim > most / (batch * tokens)) return GS_ERR_INVALID_ARGUMENT;
    if (!pos || !freq || (heads_q > 0 && (!q->data || !q_out->data)) || (heads_k > 0 && (!k->data || !k_out->data)))
        return GS_ERR_INVALID_ARGUMENT;
    RopeArgs a{};
    a.batch = batch;
    a.tokens = tokens;
    a.stride_pos_b = stride_pos_b;
    a.heads_q = heads_q;
    a.heads_k = heads_k;
    a.half = dim / 2;
    a.p0 = pairs[0];
    a.p1 = pairs[1];
    a.p2 = pairs[2];
    a.interleaved = interleaved != 0;
    a.inverse = inverse != 0;
    const int e = elem_bytes(dtype), vec = 16 / e;
    const bool wide = a.half % vec == 0 && (heads_q == 0 || (rows_aligned(q, batch, tokens, heads_q, e, 16) &&
                                                             rows_aligned(q_out, batch, tokens, heads_q, e, 16))) &&
                      (heads_k == 0 || (rows_aligned(k, batch, tokens, heads_k, e, 16) &&
                                        rows_aligned(k_out, batch, tokens, heads_k, e, 16)));
    const hipStream_t s = (hipStream_t)stream;
    switch (dtype) {
        case GS_F32:
            return wide ? rope_launch<float, 4>(q, k, q_out, k_out, pos, freq, a, s)
                        : rope_launch<float, 1>(q, k, q_out, k_out, pos, freq, a, s);
        case GS_F16:
            return wide ? rope_launch<f16, 8>(q, k, q_out, k_out, pos, freq, a, s)
                        : rope_launch<f16, 1>(q, k, q_out, k_out, pos, freq, a, s);
        default:
            return wide ? rope_launch<bf16, 8>(q, k, q_out, k_out, pos, freq, a, s)
                        : rope_launch<bf16, 1>(q, k, q_out, k_out, pos, freq, a, s);
    }
}
