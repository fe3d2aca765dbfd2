// gs_block_summary and gs_block_select: 8-bit means of key blocks, and the
// blocks each group of queries attends to.
//
// Everything up to the score's one rounding is whole-number arithmetic: a
// mean of 64 keys in fixed point, 8 bits of it and a power-of-two exponent,
// an integer dot product below 2^21. So the ranking is the same whatever the
// order of the sums, and near-ties cannot flip between runs or variants. The
// choice costs one read of q and k (HBM-bound) plus blocks x dim byte
// products per group, 1 / 128 of the attention's own.
#include "tokens.h"

namespace gs {

constexpr int SEL_THREADS = 256;

__device__ __forceinline__ int to_fixed(float x)
{
    // v_med3 / max / min return the number when the other is NaN: NaN -> 0 explicitly
    const float y = rintf(x * 256.f);
    return y == y ? (int)fminf(fmaxf(y, -32768.f), 32768.f) : 0;
}

// e of the 8-bit form from the largest magnitude of the sums.
__device__ __forceinline__ int shift_of(int largest)
{
    const int bits = largest == 0 ? 0 : 32 - __builtin_clz((unsigned)largest);
    return bits > 7 ? bits - 7 : 0;
}

__device__ __forceinline__ int to_eight(int s, int e) { return min(127, (s + ((1 << e) >> 1)) >> e); }

struct SumArgs {
    int64_t tokens, block0, blocks;
    int32_t batch, heads, dim;
};

// 16-byte chunks of a row: CH elements.
template <typename T>
struct Chunk {
    static constexpr int N = 16 / sizeof(T);
};

// Sum of fixed-point elements of rows [r0, r1) of chunk c, rows r0 + first,
// + step, ...
template <typename T>
__device__ __forceinline__ void sum_rows(const T* base, int64_t row_stride, int r0, int r1, int first, int step, int c,
                                         int (&acc)[Chunk<T>::N])
{
    constexpr int N = Chunk<T>::N;
#pragma unroll 4
    for (int r = r0 + first; r < r1; r += step) {
        float x[N];
        load_f32<T, N>(base + r * row_stride + c * N, x);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += to_fixed(x[i]);
    }
}

// One workgroup per (batch, head, block): 256 threads = chunks x row slices.
template <typename T>
__global__ __launch_bounds__(SEL_THREADS) void k_block_summary(View<const T> k, const int32_t* __restrict__ kv_len,
                                                               View<int8_t> sum8, View<float> scale,
                                                               const SumArgs a)
{
    constexpr int N = Chunk<T>::N;
    __shared__ int s_sum[256];
    __shared__ int s_max;
    const int64_t id = blockIdx.x;
    const int64_t blk = a.block0 + id % a.blocks;
    const int64_t bh = id / a.blocks;
    const int64_t b = bh / a.heads, h = bh - b * a.heads;
    int64_t len = kv_len ? kv_len[b] : a.tokens;
    len = len < 0 ? 0 : (len > a.tokens ? a.tokens : len);
    const int64_t t0 = blk * GS_KEY_BLOCK;
    const int n = (int)(len - t0 < 0 ? 0 : (len - t0 < GS_KEY_BLOCK ? len - t0 : GS_KEY_BLOCK));
    for (int i = threadIdx.x; i < 256; i += SEL_THREADS) s_sum[i] = 0;
    if (threadIdx.x == 0) s_max = 0;
    __syncthreads();
    const int chunks = a.dim / N, slices = SEL_THREADS / chunks;
    const int c = threadIdx.x % chunks, slice = threadIdx.x / chunks;
    if (slice < slices) {
        int acc[N] = {};
        sum_rows<T>(k.at(b, t0, h), k.st, 0, n, slice, slices, c, acc);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (n > slice) atomicAdd(&s_sum[c * N + i], acc[i]);  // integers: any order
    }
    __syncthreads();
    const int d = threadIdx.x;
    const int v = d < a.dim ? s_sum[d] : 0;
    const int m = wave_max_int(abs(v));
    if ((threadIdx.x & 63) == 0) atomicMax(&s_max, m);
    __syncthreads();
    const int e = shift_of(s_max);
    if (d < a.dim) sum8.at(b, blk, h)[d] = (int8_t)to_eight(v, e);
    if (threadIdx.x == 0) *scale.at(b, blk, h) = ldexpf(1.f / (float)(n > 0 ? n : 1), e);
}

struct SelArgs {
    int64_t tokens_q, tokens_k, groups, blocks;
    int32_t heads_q, heads_k, dim, causal, top;
};

// Order-preserving map of finite floats to uint32 (never 0 or 0xffffffff).
__device__ __forceinline__ uint32_t rank_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One workgroup per (batch, query head, group). Dynamic LDS: the blocks' keys.
template <typename T>
__global__ __launch_bounds__(SEL_THREADS) void k_block_select(View<const T> q, View<const int8_t> sum8,
                                                              View<const float> scale,
                                                              const int32_t* __restrict__ kv_len,
                                                              int32_t* __restrict__ list, const SelArgs a)
{
    constexpr int N = Chunk<T>::N;
    extern __shared__ uint32_t s_key[];
    __shared__ int s_sum[256];
    __shared__ int s_max;
    __shared__ alignas(16) int8_t s_q[256];
    __shared__ uint32_t s_hist[256];
    __shared__ uint32_t s_pick[2];
    __shared__ uint32_t s_cnt[2][SEL_THREADS / 64];
    const int64_t id = blockIdx.x;
    const int64_t bh = id / a.groups, g = id - bh * a.groups;
    const int64_t b = bh / a.heads_q, h = bh - b * a.heads_q;
    const int64_t hk = h / (a.heads_q / a.heads_k);
    int64_t len = kv_len ? kv_len[b] : a.tokens_k;
    len = len < 0 ? 0 : (len > a.tokens_k ? a.tokens_k : len);
    const int64_t t0 = g * GS_QUERY_GROUP;
    const int n = (int)(a.tokens_q - t0 < GS_QUERY_GROUP ? a.tokens_q - t0 : GS_QUERY_GROUP);
    int32_t* out = list + id * a.top;
    // positions of the group, and the blocks it sees
    const int64_t low = t0 + len - a.tokens_q, high = low + n - 1;
    int64_t seen = len;
    if (a.causal && high + 1 < seen) seen = high + 1;
    const int64_t visible = seen > 0 ? (seen + GS_KEY_BLOCK - 1) / GS_KEY_BLOCK : 0;
    const int64_t held0 = a.causal ? (low > 0 ? low : 0) / GS_KEY_BLOCK : visible;
    if (visible <= a.top) {  // all of them: nothing to rank
        for (int64_t i = threadIdx.x; i < a.top; i += SEL_THREADS) out[i] = i < visible ? (int32_t)i : -1;
        return;
    }
    // the group's 8-bit mean
    for (int i = threadIdx.x; i < 256; i += SEL_THREADS) s_sum[i] = 0;
    if (threadIdx.x == 0) s_max = 0;
    __syncthreads();
    const int chunks = a.dim / N, slices = SEL_THREADS / chunks;
    const int c = threadIdx.x % chunks, slice = threadIdx.x / chunks;
    if (slice < slices) {
        int acc[N] = {};
        sum_rows<T>(q.at(b, t0, h), q.st, 0, n, slice, slices, c, acc);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (n > slice) atomicAdd(&s_sum[c * N + i], acc[i]);
    }
    __syncthreads();
    const int d = threadIdx.x;
    const int v = d < a.dim ? s_sum[d] : 0;
    const int m = wave_max_int(abs(v));
    if ((threadIdx.x & 63) == 0) atomicMax(&s_max, m);
    __syncthreads();
    if (d < a.dim) s_q[d] = (int8_t)to_eight(v, shift_of(s_max));
    __syncthreads();
    // scores of the visible blocks
    const int8_t* keys = sum8.at(b, 0, hk);
    const float* scales = scale.at(b, 0, hk);
    const int words = a.dim / 8;
    for (int64_t i = threadIdx.x; i < visible; i += SEL_THREADS) {
        const uint2* row = (const uint2*)(keys + i * sum8.st);
        int dot = 0;
#pragma unroll 4
        for (int w = 0; w < words; ++w) {
            const uint2 x = row[w], y = ((const uint2*)s_q)[w];
            dot = __builtin_amdgcn_sdot4((int)x.x, (int)y.x, dot, false);
            dot = __builtin_amdgcn_sdot4((int)x.y, (int)y.y, dot, false);
        }
        // the product's one rounding; + 0 turns -0 into 0, which ties with it
        const float s = (float)dot * scales[i * scale.st] + 0.f;
        s_key[i] = i >= held0 ? 0xffffffffu : rank_key(s);
    }
    // the top-th largest key, 8 bits at a time
    uint32_t prefix = 0, want = (uint32_t)a.top;
    for (int shift = 24; shift >= 0; shift -= 8) {
        s_hist[threadIdx.x] = 0;
        __syncthreads();
        for (int64_t i = threadIdx.x; i < visible; i += SEL_THREADS) {
            const uint32_t x = s_key[i];
            if (shift == 24 || (x >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_hist[(x >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (threadIdx.x < 64) {
            // lane t holds the four bins 255 - 4t .. 252 - 4t, largest first
            uint32_t bin[4], sum = 0;
            for (int i = 0; i < 4; ++i) sum += bin[i] = s_hist[255 - (threadIdx.x * 4 + i)];
            uint32_t before = sum;
            for (int off = 1; off < 64; off <<= 1) {
                const uint32_t y = __shfl_up(before, off);
                if ((int)threadIdx.x >= off) before += y;
            }
            before -= sum;
            for (int i = 0; i < 4; ++i) {
                if (before < want && before + bin[i] >= want) {
                    s_pick[0] = 255u - (threadIdx.x * 4 + i);
                    s_pick[1] = want - before;
                }
                before += bin[i];
            }
        }
        __syncthreads();
        prefix |= s_pick[0] << shift;
        want = s_pick[1];
    }
    // keys above `prefix` are all in, of those equal to it the `want` lowest
    // blocks; each thread holds a run of blocks, so ids come out ascending
    const int64_t per = (visible + SEL_THREADS - 1) / SEL_THREADS;
    const int64_t lo = threadIdx.x * per, hi = lo + per < visible ? lo + per : visible;
    uint32_t above = 0, equal = 0;
    for (int64_t i = lo; i < hi; ++i) {
        above += s_key[i] > prefix;
        equal += s_key[i] == prefix;
    }
    uint32_t ia = above, ie = equal;
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t x = __shfl_up(ia, off), y = __shfl_up(ie, off);
        if ((int)lane_id() >= off) ia += x, ie += y;
    }
    const int wave = threadIdx.x >> 6;
    if (lane_id() == 63) s_cnt[0][wave] = ia, s_cnt[1][wave] = ie;
    __syncthreads();
    ia -= above;
    ie -= equal;
    for (int w = 0; w < wave; ++w) ia += s_cnt[0][w], ie += s_cnt[1][w];
    for (int64_t i = lo; i < hi; ++i) {
        const uint32_t x = s_key[i];
        if (x > prefix) {
            out[ia + min(ie, want)] = (int32_t)i;
            ++ia;
        } else if (x == prefix) {
            if (ie < want) out[ia + ie] = (int32_t)i;
            ++ie;
        }
    }
}

template <typename T>
static gs_status summary_launch(const gs_tokens* k, const int32_t* kv_len, const gs_tokens* sum8,
                                const gs_tokens* scale, const SumArgs& a, hipStream_t s)
{
    hipLaunchKernelGGL((k_block_summary<T>), dim3((unsigned)((int64_t)a.batch * a.heads * a.blocks)), dim3(SEL_THREADS),
                       0, s, view_of<const T>(k), kv_len, view_of<int8_t>(sum8), view_of<float>(scale), a);
    GS_CHECK_LAUNCH();
    return GS_OK;
}

template <typename T>
static gs_status select_launch(const gs_tokens* q, const gs_tokens* sum8, const gs_tokens* scale, const int32_t* kv_len,
                               int32_t* list, int64_t lists, const SelArgs& a, hipStream_t s)
{
    // keys of every block that can be visible; above 64 KiB the kernel asks for more LDS
    const size_t lds = (size_t)a.blocks * 4;
    if (lds > 65536 - 8192 &&
        hipFuncSetAttribute((const void*)k_block_select<T>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) != hipSuccess)
        return GS_ERR_HIP;
    hipLaunchKernelGGL((k_block_select<T>), dim3((unsigned)lists), dim3(SEL_THREADS), lds, s, view_of<const T>(q),
                       view_of<const int8_t>(sum8), view_of<const float>(scale), kv_len, list, a);
    GS_CHECK_LAUNCH();
    return GS_OK;
}

}  // namespace gs

extern "C" {

gs_status gs_block_summary(const gs_tokens* k, int64_t batch, int64_t tokens, int32_t heads, int32_t dim,
                           int32_t dtype, const int32_t* kv_len, int64_t block0, int64_t blocks,
                           const gs_tokens* sum8, const gs_tokens* scale, void* stream)
{
    using namespace gs;
    const int64_t most = (int64_t)1 << 40;
    if (!k || !sum8 || !scale || batch < 0 || tokens < 0 || tokens > most || heads < 0 || dim < 8 || dim > 256 || (dim & 7) ||
        !dtype_ok(dtype) || block0 < 0 || blocks < 0)
        return GS_ERR_INVALID_ARGUMENT;
    const int64_t all = (tokens + GS_KEY_BLOCK - 1) / GS_KEY_BLOCK;
    if (block0 > all || blocks > all - block0) return GS_ERR_INVALID_ARGUMENT;
    if (batch == 0 || heads == 0 || blocks == 0) return GS_OK;
    if (!k->data || !sum8->data || !scale->data) return GS_ERR_INVALID_ARGUMENT;
    const int64_t grid_most = (int64_t)1 << 23;  // 256 threads each, below 2^32 in all
    if (batch > grid_most || heads > grid_most / batch || blocks > grid_most / (batch * heads))
        return GS_ERR_UNSUPPORTED;
    if (!rows_aligned(k, batch, tokens, heads, elem_bytes(dtype), 16)) return GS_ERR_UNSUPPORTED;
    const SumArgs a{tokens, block0, blocks, (int32_t)batch, heads, dim};
    const hipStream_t s = (hipStream_t)stream;
    switch (dtype) {
        case GS_F32: return summary_launch<float>(k, kv_len, sum8, scale, a, s);
        case GS_F16: return summary_launch<f16>(k, kv_len, sum8, scale, a, s);
        default: return summary_launch<bf16>(k, kv_len, sum8, scale, a, s);
    }
}

gs_status gs_block_select(const gs_tokens* q, const gs_tokens* sum8, const gs_tokens* scale, int64_t batch,
                          int64_t tokens_q, int64_t tokens_k, int32_t heads_q, int32_t heads_k, int32_t dim,
                          int32_t dtype, const int32_t* kv_len, int32_t causal, int32_t top, int32_t* list,
                          void* stream)
{
    using namespace gs;
    if (!q || !sum8 || !scale || batch < 0 || tokens_q < 0 || tokens_k < 0 || tokens_k > GS_MAX_SELECT_TOKENS || heads_q < 1 ||
        heads_k < 1 || heads_q % heads_k != 0 || dim < 8 || dim > 256 || (dim & 7) || !dtype_ok(dtype) || top < 1 ||
        top > 32768 || tokens_q > ((int64_t)1 << 40))
        return GS_ERR_INVALID_ARGUMENT;
    const int64_t groups = (tokens_q + GS_QUERY_GROUP - 1) / GS_QUERY_GROUP;
    const int64_t blocks = (tokens_k + GS_KEY_BLOCK - 1) / GS_KEY_BLOCK;
    if (batch == 0 || groups == 0) return GS_OK;
    if (!q->data || !list || (blocks > 0 && (!sum8->data || !scale->data))) return GS_ERR_INVALID_ARGUMENT;
    const int64_t grid_most = (int64_t)1 << 23;
    if (batch > grid_most || heads_q > grid_most / batch || groups > grid_most / (batch * heads_q))
        return GS_ERR_UNSUPPORTED;
    if (!rows_aligned(q, batch, tokens_q, heads_q, elem_bytes(dtype), 16)) return GS_ERR_UNSUPPORTED;
    if (!rows_aligned(sum8, batch, blocks, heads_k, 1, 8)) return GS_ERR_UNSUPPORTED;
    const SelArgs a{tokens_q, tokens_k, groups, blocks, heads_q, heads_k, dim, causal != 0, top};
    const hipStream_t s = (hipStream_t)stream;
    const int64_t lists = batch * heads_q * groups;
    switch (dtype) {
        case GS_F32: return select_launch<float>(q, sum8, scale, kv_len, list, lists, a, s);
        case GS_F16: return select_launch<f16>(q, sum8, scale, kv_len, list, lists, a, s);
        default: return select_launch<bf16>(q, sum8, scale, kv_len, list, lists, a, s);
    }
}

}  // extern "C"
