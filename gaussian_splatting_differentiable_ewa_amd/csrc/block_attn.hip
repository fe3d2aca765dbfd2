// gs_block_attn_fwd: softmax attention of query groups over their listed key
// blocks.
#include "block_attn.h"

namespace gs {

// Softmax state of a wave's 32 queries (one per lane column).
template <int D>
struct Online {
    float m, l;  // running maximum (scaled to base 2) and this lane half's sum
    acc16 o[D / 32];
    __device__ __forceinline__ void init()
    {
        m = -INFINITY;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = zero16();
    }
};

// The running maximum is renewed, and sums and outputs rescaled, only when a
// score exceeds it by more than 2^8: until then probabilities are at most 256
// instead of 1, which neither their type nor the fp32 sums notice. With the
// maximum renewed at every rise some of the 32 queries rose at nearly every
// block, at 64 multiplications a lane.
constexpr float RISE = 8.f;

// A sum of zero is a query that saw no key; a NaN (from its own row or a key it
// sees) is none, and goes on.
__device__ __forceinline__ float inverse_of(float sum) { return sum == 0.f ? 0.f : 1.f / sum; }
__device__ __forceinline__ float lse_of(float m, float sum) { return sum == 0.f ? -INFINITY : (m + log2f(sum)) * LN2; }

// One block of 64 keys. Probabilities are rounded to the inputs' type for their
// product with the values, which the matrix unit takes in that type; their sum
// is of the unrounded ones, so the roundings average out instead of shifting a
// row. At 510 blocks of 64, 32 listed, dim 128, bf16: out is 2.3e-3 of its norm
// off, 1.66e-3 of which is its own rounding.
// limit is the number of keys, counted from the block's first, that this lane's
// query sees (>= 64: all of them).
template <typename T, int D, bool MASKED>
__device__ __forceinline__ void attend_block(const T* kt, const T* vt, const typename Mma<T>::v8 (&q)[D / 16],
                                             Online<D>& st, float c, int limit)
{
    const int hi = lane_id() >> 5;
    acc16 s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        s[t] = zero16();
#pragma unroll
        for (int k = 0; k < D / 16; ++k) s[t] = Mma<T>::mma(read_rows<T, D>(kt, t * 32, k), q[k], s[t]);
    }
    interleave<D / 8, D / 8, 4>();
    if constexpr (MASKED) {
        const int rows = limit - 4 * hi;  // against constants: no registers for the rows
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[t][i] = t * 32 + c_row(i, 0) < rows ? s[t][i] : -INFINITY;
    }
    float mx = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[t][i]);
    mx = fmaxf(mx, __shfl_xor(mx, 32)) * c;
    if (__any(mx > st.m + RISE)) {
        const float m = fmaxf(st.m, mx);
        const float f = m == -INFINITY ? 1.f : exp2_fast(st.m - m);
        st.m = m;
        st.l *= f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) st.o[i][j] *= f;
    }
    const float ms = st.m == -INFINITY ? 0.f : st.m;  // nothing seen so far: every p is 0
    typename Mma<T>::v8 p[4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            s[t][i] = exp2_fast(fmaf(s[t][i], c, -ms));
            st.l += s[t][i];
        }
        p[2 * t] = as_operand<T>(s[t], 0);
        p[2 * t + 1] = as_operand<T>(s[t], 1);
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) st.o[i] = Mma<T>::mma(read_cols<T, D>(vt, k * 16, i * 32), p[k], st.o[i]);
    interleave<D / 4, D / 8, 8>();
}

// Many queries: a workgroup per (batch, head, group), four waves of 32
// queries, the listed blocks one after the other through two LDS stages.
// A block is read once for 128 queries (128 x 64 x 4 x dim operations for 64 x
// 2 x dim x 2 bytes: 128 a byte, from L2 mostly), and two workgroups a CU (four
// at dim 64) let one wave's exponentials run behind another's matrix
// instructions. Per block and wave at dim 128: 32 matrix instructions of 32
// cycles each and 32 exponentials, maxima, sums and roundings a lane beside
// them; at dim 64 half the former and all of the latter, which then bound it.
// Measured: dim 128, 16 heads, 255 groups, 32 blocks each 578 us, 950 TFLOP/s
// (656 after seconds of load, where the clocks fall; large library product:
// 1350; matrix unit busy 47 %, vector instructions in 45 % of the cycles, no LDS
// bank conflicts); dim 64, 16 heads on 4 key heads, 254 groups of 16 blocks,
// causal 170 to 195 us (39 % and 73 %).
template <typename T, int D>
__device__ __forceinline__ void attn_fwd(T (&s_tile)[2][2][Tile<D>::ELEMS], const View<const T>& q, const View<const T>& k,
                                         const View<const T>& v, const int32_t* __restrict__ lists,
                                         const int32_t* __restrict__ kv_len, const View<T>& out,
                                         float* __restrict__ lse, const AttnArgs& a)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id(), hi = lane >> 5;
    const int64_t id = xcd_contiguous(blockIdx.x, gridDim.x);
    const int64_t bh = id / a.groups, g = id - bh * a.groups;
    const int64_t b = bh / a.heads_q, h = bh - b * a.heads_q, hk = h / (a.heads_q / a.heads_k);
    const int32_t* list = lists + id * a.top;
    const int64_t len = seq_len(kv_len, b, a.tokens_k);
    const int64_t i0 = g * QG, i = i0 + wave * 32 + (lane & 31);
    // keys the lane's query and the group's last and first query see
    const int64_t past = len - a.tokens_q;
    const int64_t end = i0 + QG < a.tokens_q ? i0 + QG : a.tokens_q;
    const int64_t mine = a.causal && past + i + 1 < len ? past + i + 1 : len;
    const int64_t most = a.causal && past + end < len ? past + end : len;
    const int64_t least = a.causal && past + i0 + 1 < len ? past + i0 + 1 : len;
    const int64_t visible = most > 0 ? (most + KB - 1) / KB : 0;
    const float c = a.scale * LOG2E;

    typename Mma<T>::v8 qf[D / 16];
    load_cols<T, D>(q.at(b, i < a.tokens_q ? i : a.tokens_q - 1, h), qf);
    Online<D> st;
    st.init();
    const T* kb = k.at(b, 0, hk);
    const T* vb = v.at(b, 0, hk);
    const TileLoad<T, D, 4> load_k(k.st), load_v(v.st);
    ListWalk walk(list, a.top, visible);
    int blk = walk.next();
    if (blk >= 0) {
        load_k(s_tile[0][0], kb, (int64_t)blk * KB, len - 1, wave);
        load_v(s_tile[0][1], vb, (int64_t)blk * KB, len - 1, wave);
    }
    auto step = [&](int S, auto masked) __attribute__((always_inline)) {
        const int next = walk.next();
        wait_loads();
        __syncthreads();  // the stage is whole, and the other one is read out
        if (next >= 0) {
            load_k(s_tile[S ^ 1][0], kb, (int64_t)next * KB, len - 1, wave);
            load_v(s_tile[S ^ 1][1], vb, (int64_t)next * KB, len - 1, wave);
        }
        const int64_t k0 = (int64_t)blk * KB, rest = mine - k0;
        const int limit = (int)(rest < 0 ? 0 : (rest < KB ? rest : KB));
        attend_block<T, D, decltype(masked)::value>(s_tile[S][0], s_tile[S][1], qf, st, c, limit);
        blk = next;
    };
    walk_blocks(step, [&] { return blk >= 0; }, [&] { return (int64_t)blk * KB + KB > least; });
    if (i >= a.tokens_q) return;
    const float l = st.l + __shfl_xor(st.l, 32);
    const float inv = inverse_of(l);
    T* o = out.at(b, i, h);
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            store4<T>(o + t * 32 + r * 8 + hi * 4, st.o[t][4 * r] * inv, st.o[t][4 * r + 1] * inv,
                      st.o[t][4 * r + 2] * inv, st.o[t][4 * r + 3] * inv);
    if (hi == 0) lse[bh * a.tokens_q + i] = lse_of(st.m, l);
}

template <typename T, int D>
__global__ __launch_bounds__(ATT_THREADS, D == 64 ? 4 : 2) void k_attn_fwd(View<const T> q, View<const T> k,
                                                                          View<const T> v, const int32_t* lists,
                                                                          const int32_t* kv_len, View<T> out, float* lse,
                                                                          const AttnArgs a)
{
    __shared__ alignas(16) T s_tile[2][2][Tile<D>::ELEMS];
    attn_fwd<T, D>(s_tile, q, k, v, lists, kv_len, out, lse, a);
}

// Few queries: a workgroup per 32 queries and split of their list; its four
// waves take the split's entries in turn, each with its own tiles, and join
// at the end (the softmax states of disjoint key sets add after rescaling to
// the common maximum). With more than one split the joined states go to the
// workspace and k_attn_join ends the work.
// Bound by latency: one query, 16 heads of dim 128, 32 blocks: 8.5 us and 2.7
// for the join (16 MB of keys and values, 3.3 us at the copy rate).
template <typename T, int D>
__global__ __launch_bounds__(ATT_THREADS, 1) void k_attn_few(View<const T> q, View<const T> k, View<const T> v,
                                                             const int32_t* __restrict__ lists,
                                                             const int32_t* __restrict__ kv_len, View<T> out,
                                                             float* __restrict__ lse, float* __restrict__ part,
                                                             const AttnArgs a)
{
    __shared__ alignas(16) T s_tile[4][2][Tile<D>::ELEMS];
    __shared__ float s_m[4][32], s_l[4][32];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id(), hi = lane >> 5;
    const int64_t tiles = (a.tokens_q + 31) / 32;
    const int64_t unit = blockIdx.x / a.splits;
    const int split = (int)(blockIdx.x - unit * a.splits);
    const int64_t bh = unit / tiles, tile = unit - bh * tiles;
    const int64_t b = bh / a.heads_q, h = bh - b * a.heads_q, hk = h / (a.heads_q / a.heads_k);
    const int64_t i0 = tile * 32, i = i0 + (lane & 31);
    const int32_t* list = lists + (bh * a.groups + i0 / QG) * a.top;
    const int64_t len = seq_len(kv_len, b, a.tokens_k), past = len - a.tokens_q;
    const int64_t end = i0 + 32 < a.tokens_q ? i0 + 32 : a.tokens_q;
    const int64_t mine = a.causal && past + i + 1 < len ? past + i + 1 : len;
    const int64_t most = a.causal && past + end < len ? past + end : len;
    const int64_t least = a.causal && past + i0 + 1 < len ? past + i0 + 1 : len;
    const int64_t visible = most > 0 ? (most + KB - 1) / KB : 0;
    const float c = a.scale * LOG2E;

    typename Mma<T>::v8 qf[D / 16];
    load_cols<T, D>(q.at(b, i < a.tokens_q ? i : a.tokens_q - 1, h), qf);
    Online<D> st;
    st.init();
    const T* kb = k.at(b, 0, hk);
    const T* vb = v.at(b, 0, hk);
    const TileLoad<T, D, 1> load_k(k.st), load_v(v.st);
    ListWalk walk(list, a.top, visible, split * 4 + wave, 4 * a.splits);
    for (int blk = walk.next(); blk >= 0; blk = walk.next()) {
        const int64_t k0 = (int64_t)blk * KB, rest = mine - k0;
        // the wave's own reads of the tile's last contents are done: their
        // results were used
        load_k(s_tile[wave][0], kb, k0, len - 1, 0);
        load_v(s_tile[wave][1], vb, k0, len - 1, 0);
        wait_loads();
        const int limit = (int)(rest < 0 ? 0 : (rest < KB ? rest : KB));
        // one form for both kinds of block: a wave has few
        attend_block<T, D, true>(s_tile[wave][0], s_tile[wave][1], qf, st, c, limit);
    }
    const float l = st.l + __shfl_xor(st.l, 32);
    if (hi == 0) s_m[wave][lane] = st.m, s_l[wave][lane] = l;
    __syncthreads();  // also: every wave is done with its tiles
    // the waves' outputs side by side in the tiles' memory: [wave][D][32]
    float* s_o = (float*)&s_tile[0][0][0];
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) s_o[(wave * D + t * 32 + c_row(r, hi)) * 32 + (lane & 31)] = st.o[t][r];
    __syncthreads();
    const int col = threadIdx.x & 31;
    float m = -INFINITY, f[4], total = 0.f;
    for (int w = 0; w < 4; ++w) m = fmaxf(m, s_m[w][col]);
    for (int w = 0; w < 4; ++w) {
        f[w] = m == -INFINITY ? 0.f : exp2_fast(s_m[w][col] - m);
        total += f[w] * s_l[w][col];
    }
    const int64_t at = i0 + col;
    if (at >= a.tokens_q) return;
    const float inv = inverse_of(total);
    constexpr int PER = D / 8;  // dimensions of one thread
    const int d0 = (threadIdx.x >> 5) * PER;
    float x[PER];
#pragma unroll
    for (int d = 0; d < PER; ++d) {
        x[d] = 0.f;
        for (int w = 0; w < 4; ++w) x[d] += f[w] * s_o[(w * D + d0 + d) * 32 + col];
    }
    if (a.splits == 1) {
        T* o = out.at(b, at, h) + d0;
#pragma unroll
        for (int d = 0; d < PER; d += 4) store4<T>(o + d, x[d] * inv, x[d + 1] * inv, x[d + 2] * inv, x[d + 3] * inv);
        if (d0 == 0) lse[bh * a.tokens_q + at] = lse_of(m, total);
    } else {
        float* p = part + ((bh * a.tokens_q + at) * a.splits + split) * (D + 4);
#pragma unroll
        for (int d = 0; d < PER; d += 4) *(float4*)(p + 4 + d0 + d) = make_float4(x[d], x[d + 1], x[d + 2], x[d + 3]);
        if (d0 == 0) p[0] = m, p[1] = total;
    }
}

// Joins the splits of one query: D / 4 threads a query.
template <typename T, int D>
__global__ __launch_bounds__(ATT_THREADS) void k_attn_join(const float* __restrict__ part, int64_t queries, View<T> out,
                                                           float* __restrict__ lse, const AttnArgs a)
{
    constexpr int TH = D / 4;
    const int64_t row = (int64_t)blockIdx.x * (ATT_THREADS / TH) + threadIdx.x / TH;
    if (row >= queries) return;
    const int d0 = threadIdx.x % TH * 4;
    const float* p = part + row * a.splits * (D + 4);
    float m = -INFINITY, total = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    // eight splits at a time, all their loads in flight at once
    for (int s0 = 0; s0 < a.splits; s0 += 8) {
        float2 ml[8];
        float4 y[8];
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const float* ps = p + (s0 + s < a.splits ? s0 + s : a.splits - 1) * (D + 4);
            ml[s] = *(const float2*)ps;
            y[s] = *(const float4*)(ps + 4 + d0);
        }
        float most = m;
#pragma unroll
        for (int s = 0; s < 8; ++s) most = s0 + s < a.splits ? fmaxf(most, ml[s].x) : most;
        // nothing seen so far: factors of zero (not skipped: a sum may be NaN)
        const float ref = most == -INFINITY ? 0.f : most, old = exp2_fast(m - ref);
        total *= old;
        x.x *= old, x.y *= old, x.z *= old, x.w *= old;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
            const float f = s0 + s < a.splits ? exp2_fast(ml[s].x - ref) : 0.f;
            total = fmaf(f, ml[s].y, total);
            x.x = fmaf(f, y[s].x, x.x), x.y = fmaf(f, y[s].y, x.y), x.z = fmaf(f, y[s].z, x.z), x.w = fmaf(f, y[s].w, x.w);
        }
        m = most;
    }
    const float inv = inverse_of(total);
    const int64_t bh = row / a.tokens_q, i = row - bh * a.tokens_q, b = bh / a.heads_q, h = bh - b * a.heads_q;
    store4<T>(out.at(b, i, h) + d0, x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    if (d0 == 0) lse[row] = lse_of(m, total);
}

gs_status attn_check(int64_t batch, int64_t tokens_q, int64_t tokens_k, int32_t heads_q, int32_t heads_k, int32_t dim,
                     int32_t dtype, int32_t top, float sm_scale)
{
    const int64_t most = (int64_t)1 << 40;
    if (batch < 0 || tokens_q < 0 || tokens_k < 0 || tokens_q > most || tokens_k > ((int64_t)1 << 36) || heads_q < 1 ||
        heads_k < 1 || heads_q % heads_k != 0 || dim < 1 || !dtype_ok(dtype) || top < 1 || !(sm_scale > 0.f) ||
        !(sm_scale < INFINITY))
        return GS_ERR_INVALID_ARGUMENT;
    if ((dim != 64 && dim != 128) || dtype == GS_F32) return GS_ERR_UNSUPPORTED;
    // one workgroup of 256 threads per unit of 32 queries, of 512 per 64 keys: below 2^32 threads in all
    const int64_t units = ((int64_t)1 << 23) - 1;
    const int64_t per = std::max((tokens_q + 31) / 32, (tokens_k + KB - 1) / KB);
    if (batch > units || (batch > 0 && heads_q > units / batch) ||
        (batch > 0 && per > units / (batch * heads_q)))
        return GS_ERR_UNSUPPORTED;
    return GS_OK;
}

// The split of few queries: while a workgroup per group would leave most of
// the 256 CUs idle. It reads each block for 32 queries where the other kernel
// reads it for 128, so it must not be kept longer. Whole calls in us, one
// workgroup per group against this one, at lists of 4, 16 and 64 blocks:
//   dim 128, 48 groups   15/15  26/28  86/60    dim 64,  96 groups  15/15  22/15  73/42
//            64 groups   15/15  26/18  86/52            128 groups  15/15  22/16  74/46
//            92 groups   15/17  26/33  87/90            188 groups  15/15  23/24  74/66
//           128 groups   15/20  26/35  86/92            256 groups  15/16  24/29  74/80
// A limit on groups alone cannot suit every length; where it errs it costs up to
// a third (92 groups, 16 blocks).
struct Plan {
    bool few;
    int splits;
};

static Plan attn_plan(int64_t batch, int64_t tokens_q, int32_t heads_q, int32_t dim, int32_t top)
{
    const int64_t groups = (tokens_q + QG - 1) / QG, tiles = (tokens_q + 31) / 32, bh = batch * heads_q;
    Plan p{};
    p.few = bh * groups < (dim == 128 ? 96 : 192);
    p.splits = 1;
    if (p.few) {
        const int64_t want = (256 + bh * tiles - 1) / (bh * tiles), most = (top + 3) / 4;
        p.splits = (int)std::max<int64_t>(1, std::min(want, most));
    }
    return p;
}

template <typename T, int D>
static gs_status attn_fwd_launch(const gs_tokens* q, const gs_tokens* k, const gs_tokens* v, const int32_t* list,
                                 const int32_t* kv_len, const gs_tokens* out, float* lse, float* part, int64_t batch,
                                 AttnArgs a, const Plan& plan, hipStream_t s)
{
    const int64_t bh = batch * a.heads_q;
    if (!plan.few) {
        hipLaunchKernelGGL((k_attn_fwd<T, D>), dim3((unsigned)(bh * a.groups)), dim3(ATT_THREADS), 0, s,
                           view_of<const T>(q), view_of<const T>(k), view_of<const T>(v), list, kv_len, view_of<T>(out),
                           lse, a);
        GS_CHECK_LAUNCH();
        return GS_OK;
    }
    const int64_t tiles = (a.tokens_q + 31) / 32;
    hipLaunchKernelGGL((k_attn_few<T, D>), dim3((unsigned)(bh * tiles * a.splits)), dim3(ATT_THREADS), 0, s,
                       view_of<const T>(q), view_of<const T>(k), view_of<const T>(v), list, kv_len, view_of<T>(out), lse,
                       part, a);
    GS_CHECK_LAUNCH();
    if (a.splits > 1) {
        hipLaunchKernelGGL((k_attn_join<T, D>), dim3(grid_for((uint64_t)(bh * a.tokens_q), ATT_THREADS / (D / 4))),
                           dim3(ATT_THREADS), 0, s, part, bh * a.tokens_q, view_of<T>(out), lse, a);
        GS_CHECK_LAUNCH();
    }
    return GS_OK;
}

}  // namespace gs

extern "C" {

size_t gs_block_attn_fwd_workspace_bytes(int64_t batch, int64_t tokens_q, int32_t heads_q, int32_t dim, int32_t top)
{
    using namespace gs;
    if (attn_check(batch, tokens_q, 0, heads_q, 1, dim, GS_BF16, top, 1.f) != GS_OK) return 0;
    if (batch == 0 || tokens_q == 0) return 0;
    const Plan p = attn_plan(batch, tokens_q, heads_q, dim, top);
    return p.splits > 1 ? (size_t)(batch * heads_q * tokens_q) * p.splits * (dim + 4) * 4 : 0;
}

gs_status gs_block_attn_fwd(const gs_tokens* q, const gs_tokens* k, const gs_tokens* v, const int32_t* list,
                            int64_t batch, int64_t tokens_q, int64_t tokens_k, int32_t heads_q, int32_t heads_k,
                            int32_t dim, int32_t dtype, const int32_t* kv_len, int32_t causal, int32_t top,
                            float sm_scale, const gs_tokens* out, float* lse, void* ws, size_t ws_bytes, void* stream)
{
    using namespace gs;
    if (!q || !k || !v || !out) return GS_ERR_INVALID_ARGUMENT;
    const gs_status st = attn_check(batch, tokens_q, tokens_k, heads_q, heads_k, dim, dtype, top, sm_scale);
    if (st != GS_OK) return st;
    if (batch == 0 || tokens_q == 0) return GS_OK;
    if (!q->data || !out->data || !lse || !list || (tokens_k > 0 && (!k->data || !v->data)))
        return GS_ERR_INVALID_ARGUMENT;
    if (!attn_view_ok(q, batch, tokens_q, heads_q) || !attn_view_ok(out, batch, tokens_q, heads_q) ||
        (tokens_k > 0 && (!attn_view_ok(k, batch, tokens_k, heads_k) || !attn_view_ok(v, batch, tokens_k, heads_k))))
        return GS_ERR_UNSUPPORTED;
    const size_t need = gs_block_attn_fwd_workspace_bytes(batch, tokens_q, heads_q, dim, top);
    if (need > 0 && (!ws || ((uintptr_t)ws & 15) || ws_bytes < need)) return GS_ERR_INVALID_ARGUMENT;
    const Plan plan = attn_plan(batch, tokens_q, heads_q, dim, top);
    const AttnArgs a{tokens_q, tokens_k, (tokens_q + QG - 1) / QG, (tokens_k + KB - 1) / KB, heads_q, heads_k,
                     causal != 0, top, plan.splits, sm_scale};
    const hipStream_t s = (hipStream_t)stream;
    if (dtype == GS_BF16)
        return dim == 128 ? attn_fwd_launch<bf16, 128>(q, k, v, list, kv_len, out, lse, (float*)ws, batch, a, plan, s)
                          : attn_fwd_launch<bf16, 64>(q, k, v, list, kv_len, out, lse, (float*)ws, batch, a, plan, s);
    return dim == 128 ? attn_fwd_launch<f16, 128>(q, k, v, list, kv_len, out, lse, (float*)ws, batch, a, plan, s)
                      : attn_fwd_launch<f16, 64>(q, k, v, list, kv_len, out, lse, (float*)ws, batch, a, plan, s);
}

}  // extern "C"
