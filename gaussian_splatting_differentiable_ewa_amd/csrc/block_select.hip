// gs_block_summary and gs_block_select: 8-bit means of key blocks, and the
// blocks each group of queries attends to.
//
// Everything up to the score's one rounding is whole-number arithmetic: a
// mean of 64 keys in fixed point, 8 bits of it and a power-of-two exponent,
// an integer dot product of at most 2^22 (dim 256), exact in fp32. So the
// ranking is the same whatever the order of the sums, and near-ties cannot flip
// between runs or variants. The choice costs one read of q and k (HBM-bound)
// plus blocks x dim byte products per group, 1 / 128 of the attention's own.
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
// Bound by the read of k: 32640 tokens, 16 heads of dim 128, bf16, 28.5 us,
// 4.7 TB/s.
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
    int64_t tokens_q, tokens_k, groups, blocks, lists;
    int32_t heads_q, heads_k, dim, causal, top, wide;  // wide: summary rows on 16 bytes
};

// Order-preserving map of finite floats to uint32 (never 0 or 0xffffffff).
__device__ __forceinline__ uint32_t rank_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int dot16(const uint4& x, const uint4& y, int dot)
{
    dot = __builtin_amdgcn_sdot4((int)x.x, (int)y.x, dot, false);
    dot = __builtin_amdgcn_sdot4((int)x.y, (int)y.y, dot, false);
    dot = __builtin_amdgcn_sdot4((int)x.z, (int)y.z, dot, false);
    return __builtin_amdgcn_sdot4((int)x.w, (int)y.w, dot, false);
}

// Sum over each eight consecutive lanes; all of them get it.
__device__ __forceinline__ int sum8_lanes(int x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0xb1, 0xf, 0xf, false);   // quad_perm 1,0,3,2
    x += __builtin_amdgcn_update_dpp(0, x, 0x4e, 0xf, 0xf, false);   // quad_perm 2,3,0,1
    return x + __builtin_amdgcn_update_dpp(0, x, 0x141, 0xf, 0xf, false);  // row_half_mirror
}

// Between the W waves of a list: a barrier, or nothing but order within a wave.
template <int W>
__device__ __forceinline__ void list_sync()
{
    if constexpr (W > 1) __syncthreads();
    else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// One list (batch, query head, group) per W waves: the scores stay in
// registers, KEYS a lane, block 64 W j + thread for j = 0 .. KEYS - 1, and the
// top-th largest is found bit by bit from the top by counting (ballots and
// scalar counts, no atomics: the scores of a list agree in their high bits, so
// a histogram's additions would fall on few addresses).
// Measured, dim 128, bf16: 4080 lists of 32 out of 510 blocks 48 us (reads q at
// 2.8 TB/s with the vector unit 56 % busy; waves wait 61 % of their time: mean,
// scores and counting of a list are in series, and the other lists' do not hide
// all of it); one new token against 2040 blocks,
// 16 lists 19 us, which is latency: the mean 4, the scores 5, counting and
// output 9.
template <typename T, int W, int KEYS>
__global__ __launch_bounds__(W < 4 ? 256 : 64 * W) void k_block_select(View<const T> q, View<const int8_t> sum8,
                                                                      View<const float> scale,
                                                                      const int32_t* __restrict__ kv_len,
                                                                      int32_t* __restrict__ list, const SelArgs a)
{
    constexpr int N = Chunk<T>::N, PER = W < 4 ? 4 / W : 1, THREADS = 64 * W;
    __shared__ int s_sum[PER][256];
    __shared__ int s_max[PER];
    __shared__ int s_seen[PER];
    __shared__ alignas(16) int8_t s_q[PER][256];
    __shared__ uint32_t s_cnt[2][3][16];
    __shared__ uint32_t s_start[W > 1 ? 2 * KEYS * W : 1];
    __shared__ int s_dot[W == 1 ? PER : 1][W == 1 ? 64 * KEYS : 1];
    const int which = threadIdx.x / THREADS, tid = threadIdx.x % THREADS, wave = tid >> 6;
    const int64_t first_id = (int64_t)blockIdx.x * PER;
    // past the last list: its work again, without its output
    const bool extra = first_id + which >= a.lists;
    const int64_t id = extra ? a.lists - 1 : first_id + which;
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
    const int visible = seen > 0 ? (int)((seen + GS_KEY_BLOCK - 1) / GS_KEY_BLOCK) : 0;
    const int held0 = a.causal ? (int)((low > 0 ? low : 0) / GS_KEY_BLOCK) : visible;
    const bool all = visible <= a.top;  // nothing to rank
    if (all && !extra)
        for (int i = tid; i < a.top; i += THREADS) out[i] = i < visible ? i : -1;
    if (W > 1 && all) return;  // one list a workgroup; else the waves go on together
    // the group's 8-bit mean
    for (int i = tid; i < 256; i += THREADS) s_sum[which][i] = 0;
    if (tid == 0) s_max[which] = 0, s_seen[which] = visible;
    list_sync<W>();
    const int chunks = a.dim / N, slices = THREADS / chunks;
    const int c = tid % chunks, slice = tid / chunks;
    if (slice < slices && slice < n) {
        int acc[N] = {};
        sum_rows<T>(q.at(b, t0, h), q.st, 0, n, slice, slices, c, acc);
#pragma unroll
        for (int i = 0; i < N; ++i) atomicAdd(&s_sum[which][c * N + i], acc[i]);  // integers: any order
    }
    list_sync<W>();
    int m = 0;
    for (int d = tid; d < a.dim; d += THREADS) m = max(m, abs(s_sum[which][d]));
    m = wave_max_int(m);
    if constexpr (W > 1) {
        if (lane_id() == 0) atomicMax(&s_max[0], m);
        __syncthreads();
        m = s_max[0];
    }
    const int e = shift_of(m);
    for (int d = tid; d < a.dim; d += THREADS) s_q[which][d] = (int8_t)to_eight(s_sum[which][d], e);
    list_sync<W>();
    // scores of the visible blocks; a key of 0 stands for none. Eight lanes
    // read a row, 16 bytes each at a time, so that every line is read once and
    // whole (a row per lane rereads its line for each 16 bytes once the waves'
    // rows outgrow the L1); in step x lane l's eight take row 8 (l / 8) + x,
    // whose sum lane 8 (l / 8) + x keeps.
    const int8_t* keys = sum8.at(b, 0, hk);
    const float* scales = scale.at(b, 0, hk);
    const int sub = tid & 7, words = a.wide ? a.dim / 16 : 0;
    uint32_t key[KEYS];
    bool tiled = false;
    if constexpr (W == 1) {
        // The four lists of a workgroup share their key head nearly always:
        // then its rows are read once for all four and multiplied by the
        // matrix unit, 16 rows (columns of B) by the four means (rows of A),
        // 64 dimensions at a time. (27 us of 62 by vector dot products, at 4080
        // lists of 510 blocks and dim 128.)
        __syncthreads();
        const int64_t last_id = first_id + PER - 1 < a.lists ? first_id + PER - 1 : a.lists - 1;
        const int per = a.heads_q / a.heads_k;
        tiled = a.wide && a.dim % 64 == 0 && first_id / a.groups / per == last_id / a.groups / per;
        if (tiled) {
            typedef int int4v __attribute__((ext_vector_type(4)));
            const int lane = lane_id(), part = lane >> 4, list_of = lane & 15;
            int most = 0;
            for (int w = 0; w < PER; ++w) most = max(most, s_seen[w]);
            int4v mean[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                mean[t] = t * 64 < a.dim && list_of < PER ? ((const int4v*)s_q[list_of])[t * 4 + part] : int4v{0, 0, 0, 0};
            for (int r0 = which * 16; r0 < most; r0 += PER * 16) {
                const int r = min(r0 + list_of, most - 1);
                const int4v* row = (const int4v*)(keys + r * sum8.st);
                int4v acc = {0, 0, 0, 0};
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t * 64 < a.dim) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(mean[t], row[t * 4 + part], acc, 0, 0, 0);
                // C: column = lane & 15, rows 4 (lane >> 4) + i: the four lists are in the first 16 lanes
                if (part == 0) {
#pragma unroll
                    for (int i = 0; i < PER; ++i) s_dot[i][r0 + list_of] = acc[i];
                }
            }
        }
        __syncthreads();
        if (all || extra) return;
    }
    auto score = [&](int j) __attribute__((always_inline)) -> uint32_t {
        const int first = j * THREADS + (tid & ~7);  // of the eight rows
        int kept = 0;
        if (W == 1 && tiled) {
            kept = s_dot[which][j * THREADS + tid];
        } else {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const int i = first + x;
                int dot = 0;
                if (i < visible) {
                    const int8_t* row = keys + i * sum8.st;
                    if (a.wide) {
                        for (int w = sub; w < words; w += 8)
                            dot = dot16(((const uint4*)row)[w], ((const uint4*)s_q[which])[w], dot);
                    } else {
                        for (int w = sub; w < a.dim / 8; w += 8) {
                            const uint2 p = ((const uint2*)row)[w], r = ((const uint2*)s_q[which])[w];
                            dot = __builtin_amdgcn_sdot4((int)p.x, (int)r.x, dot, false);
                            dot = __builtin_amdgcn_sdot4((int)p.y, (int)r.y, dot, false);
                        }
                    }
                }
                dot = sum8_lanes(dot);
                kept = x == sub ? dot : kept;
            }
        }
        const int i = j * THREADS + tid;
        if (i >= visible) return 0;
        // the product's one rounding; + 0 turns -0 into 0, which ties with it
        const float s = (float)kept * scales[i * scale.st] + 0.f;
        return i >= held0 ? 0xffffffffu : rank_key(s);
    };
    if constexpr (KEYS > 8) {
        // through LDS: unrolled, the steps' addresses alone would fill the registers
        __shared__ uint32_t s_key[KEYS * THREADS];
#pragma unroll 1
        for (int j = 0; j < KEYS; ++j) s_key[j * THREADS + tid] = j * THREADS < visible ? score(j) : 0;
#pragma unroll
        for (int j = 0; j < KEYS; ++j) key[j] = s_key[j * THREADS + tid];
    } else {
#pragma unroll
        for (int j = 0; j < KEYS; ++j) key[j] = j * THREADS < visible ? score(j) : 0;
    }
    // the top-th largest key: the largest value that at least `top` keys reach
    auto count = [&](uint32_t from) {
        uint32_t n = 0;
#pragma unroll
        for (int j = 0; j < KEYS; ++j)
            if (j * THREADS < visible) n += __popcll(ballot(key[j] >= from));
        return n;
    };
    const uint32_t top = (uint32_t)a.top;
    uint32_t cut = 0;
    if constexpr (W == 1) {
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t from = cut | 1u << bit, have = count(from);
            if (have < top) continue;
            cut = from;
            if (have == top) {  // these are they, with no ties to break
                --cut;
                break;
            }
        }
    } else {
        // two bits a barrier; the waves' counts are added across 16 lanes
        for (int bit = 30; bit >= 0; bit -= 2) {
            uint32_t(&cnt)[3][16] = s_cnt[bit >> 1 & 1];
#pragma unroll
            for (int k = 1; k < 4; ++k) {
                const uint32_t c1 = count(cut | (uint32_t)k << bit);
                if (lane_id() == 0) cnt[k - 1][wave] = c1;
            }
            __syncthreads();
            uint32_t sum[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                int x = (lane_id() & 15) < W ? (int)cnt[k][lane_id() & 15] : 0;
                x = sum8_lanes(x);
                sum[k] = (uint32_t)__builtin_amdgcn_readlane(x, 0) + (uint32_t)__builtin_amdgcn_readlane(x, 8);
            }
            const int k = sum[2] >= top ? 3 : (sum[1] >= top ? 2 : (sum[0] >= top ? 1 : 0));
            cut |= (uint32_t)k << bit;
            if (k > 0 && sum[k - 1] == top) {  // these are they, with no ties to break
                --cut;
                break;
            }
        }
    }
    // keys above `cut` are all in, of those equal to it the lowest blocks that
    // are wanted; ids come out in ascending order
    uint32_t above = 0, equal = 0;  // before this wave's keys of step j
    if constexpr (W == 1) {
#pragma unroll
        for (int j = 0; j < KEYS; ++j)
            if (j * THREADS < visible) above += __popcll(ballot(key[j] > cut));
    } else {
        // per (step, wave): keys above and equal, then their exclusive sums
#pragma unroll
        for (int j = 0; j < KEYS; ++j) {
            const uint32_t x = __popcll(ballot(key[j] > cut)), y = __popcll(ballot(key[j] == cut));
            if (lane_id() == 0) s_start[j * W + wave] = x, s_start[KEYS * W + j * W + wave] = y;
        }
        __syncthreads();
        if (wave < 2) {
            uint32_t* p = s_start + wave * KEYS * W;
            constexpr int ALL = KEYS * W, EACH = (ALL + 63) / 64;
            const int lane = lane_id();
            uint32_t v[EACH], sum = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i) sum += v[i] = lane * EACH + i < ALL ? p[lane * EACH + i] : 0;
            uint32_t run = sum;
            for (int off = 1; off < 64; off <<= 1) {
                const uint32_t x = __shfl_up(run, off);
                if (lane >= off) run += x;
            }
            if (wave == 0 && lane == 63) s_max[0] = (int)run;  // all above
            run -= sum;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                if (lane * EACH + i < ALL) p[lane * EACH + i] = run;
                run += v[i];
            }
        }
        __syncthreads();
        above = (uint32_t)s_max[0];
    }
    const uint32_t want = top - above;  // of the equal ones
    above = 0;
#pragma unroll
    for (int j = 0; j < KEYS; ++j) {
        if (j * THREADS >= visible) continue;
        const uint64_t is_above = ballot(key[j] > cut), is_equal = ballot(key[j] == cut);
        if constexpr (W > 1) above = s_start[j * W + wave], equal = s_start[KEYS * W + j * W + wave];
        const uint32_t ra = above + mask_rank(is_above), re = equal + mask_rank(is_equal);
        const bool mine = key[j] > cut || (key[j] == cut && re < want);
        if (mine) out[ra + min(re, want)] = j * THREADS + tid;
        above += __popcll(is_above);
        equal += __popcll(is_equal);
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

template <typename T, int W, int KEYS>
static void select_by_waves(const gs_tokens* q, const gs_tokens* sum8, const gs_tokens* scale, const int32_t* kv_len,
                            int32_t* list, const SelArgs& a, hipStream_t s)
{
    constexpr int PER = W < 4 ? 4 / W : 1;
    hipLaunchKernelGGL((k_block_select<T, W, KEYS>), dim3(grid_for((uint64_t)a.lists, PER)), dim3(W < 4 ? 256 : 64 * W), 0, s,
                       view_of<const T>(q), view_of<const int8_t>(sum8), view_of<const float>(scale), kv_len, list, a);
}

// Waves a list: 8 scores a lane, so that they stay in registers; one wave up
// to 512 blocks, sixteen where the lists are too few to fill the CUs (one new
// token, 2040 blocks, 16 lists: 18.4 us with four waves and a histogram in
// LDS) or too long for four.
template <typename T>
static gs_status select_launch(const gs_tokens* q, const gs_tokens* sum8, const gs_tokens* scale, const int32_t* kv_len,
                               int32_t* list, const SelArgs& a, hipStream_t s)
{
    if (a.blocks > 8192) select_by_waves<T, 16, 32>(q, sum8, scale, kv_len, list, a, s);
    else if (a.blocks > 2048 || (a.lists <= 256 && a.blocks > 64)) select_by_waves<T, 16, 8>(q, sum8, scale, kv_len, list, a, s);
    else if (a.blocks > 512) select_by_waves<T, 4, 8>(q, sum8, scale, kv_len, list, a, s);
    else select_by_waves<T, 1, 8>(q, sum8, scale, kv_len, list, a, s);
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
    const int64_t grid_most = (int64_t)1 << 21;  // 1024 threads each, below 2^32 in all
    if (batch > grid_most || heads_q > grid_most / batch || groups > grid_most / (batch * heads_q))
        return GS_ERR_UNSUPPORTED;
    if (!rows_aligned(q, batch, tokens_q, heads_q, elem_bytes(dtype), 16)) return GS_ERR_UNSUPPORTED;
    if (!rows_aligned(sum8, batch, blocks, heads_k, 1, 8)) return GS_ERR_UNSUPPORTED;
    const SelArgs a{tokens_q, tokens_k, groups, blocks, batch * heads_q * groups, heads_q, heads_k, dim, causal != 0, top,
                    dim % 16 == 0 && rows_aligned(sum8, batch, blocks, heads_k, 1, 16)};
    const hipStream_t s = (hipStream_t)stream;
    switch (dtype) {
        case GS_F32: return select_launch<float>(q, sum8, scale, kv_len, list, a, s);
        case GS_F16: return select_launch<f16>(q, sum8, scale, kv_len, list, a, s);
        default: return select_launch<bf16>(q, sum8, scale, kv_len, list, a, s);
    }
}

}  // extern "C"
