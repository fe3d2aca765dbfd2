// gs_block_attn_bwd: gradients of the attention over listed key blocks.
//
// Two passes without atomics, so the bits repeat: one over the query groups
// (gq, and D = sum gout out), one over the key blocks (gk, gv), which walks
// the groups that list its block. Those come from a bit matrix
// [batch][head][block][groups / 32], which the first pass sets from its lists
// (an OR: any order).
// Both passes form S and P again from lse: 7 products in all where the
// formula's 5 would need fp32 atomics on gq.
//
// Measured, dim 128, bf16, 16 heads, 255 groups of 32 blocks, 510 blocks:
// prepare 22 us, gq 830 us (3 products: 990 TFLOP/s, matrix unit busy 49 %), order 9 us,
// gk and gv 1440 us (4 products: 760 TFLOP/s, 36 %); after seconds of load 895 and 1560.
// dim 64, the same lists: 1470 us in all.
#include <algorithm>

#include "block_attn.h"

namespace gs {

// What the passes need first: the mean key of every block, fp32
// [batch][head][block][D], zero without valid keys (one wave a block: D / 8
// lanes across, the others along the keys), and a cleared bit matrix.
template <typename T, int D>
__global__ __launch_bounds__(ATT_THREADS) void k_attn_prepare(View<const T> k, const int32_t* __restrict__ kv_len,
                                                              float* __restrict__ means, uint32_t* __restrict__ bits,
                                                              int64_t words, int64_t count, const AttnArgs a)
{
    constexpr int ACROSS = D / 8, ALONG = 64 / ACROSS;
    for (int64_t i = (int64_t)blockIdx.x * ATT_THREADS + threadIdx.x; i < words; i += (int64_t)gridDim.x * ATT_THREADS)
        bits[i] = 0;
    const int64_t id = (int64_t)blockIdx.x * (ATT_THREADS / 64) + (threadIdx.x >> 6);
    if (id >= count) return;
    const int64_t bh = id / a.blocks, blk = id - bh * a.blocks, b = bh / a.heads_k, h = bh - b * a.heads_k;
    const int64_t len = seq_len(kv_len, b, a.tokens_k), rest = len - blk * KB;
    const int n = (int)(rest < 0 ? 0 : (rest < KB ? rest : KB));
    const int c = lane_id() % ACROSS, first = lane_id() / ACROSS;
    const T* base = k.at(b, blk * KB, h) + c * 8;
    float sum[8] = {};
#pragma unroll 4
    for (int r = first; r < n; r += ALONG) {
        float x[8];
        load_f32<T, 8>(base + r * k.st, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += x[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        for (int off = ACROSS; off < 64; off <<= 1) sum[e] += __shfl_xor(sum[e], off);
    if (first == 0) {
        const float inv = n > 0 ? 1.f / (float)n : 0.f;
        float* o = means + id * D + c * 8;
        *(float4*)o = make_float4(sum[0] * inv, sum[1] * inv, sum[2] * inv, sum[3] * inv);
        *(float4*)(o + 4) = make_float4(sum[4] * inv, sum[5] * inv, sum[6] * inv, sum[7] * inv);
    }
}

// gq of a group (and, for the other pass, -lse in base 2 and D of its 128
// queries, [list][2][128]): four waves of 32 queries, the listed blocks in turn.
//   dS^T = P^T (V gout^T - D),  gq^T += K^T dS^T
// D from the rounded `out` carries that rounding, an error e the same for all
// keys of a query, so gq would be off by e sum_j P_j k_j: more than all the
// other roundings together; and what the keys have in common, which cancels
// in gq, does not cancel in the roundings of dS. But the exact dS of a query
// add to zero, so with R the sum of the rounded ones gq - R c is gq's value
// for any vector c, without either error's part along c. c is the mean key as
// this wave's 32 queries weigh the blocks (from the first half of each; an
// estimate is enough). In the blocks that masks cut, where the first queries of
// a causal sequence have all their few keys and nothing averages out, dS is
// kept in two parts. D with the sum of the unrounded ones added, -e, goes to
// the other pass.
// LDS of the workgroup, in bytes: two stages of K and V, then c of the four waves.
template <typename T, int D>
struct GqLds {
    static constexpr uint32_t TILE = Tile<D>::ELEMS * sizeof(T), STAGE = 2 * TILE, MEAN = 2 * STAGE;
    static constexpr uint32_t BYTES = MEAN + 4 * D * 4;
};

template <typename T, int D>
__device__ __forceinline__ void attn_gq(char* lds, const View<const T>& go, const View<const T>& q, const View<const T>& k,
                                        const View<const T>& v, const View<const T>& out, const float* __restrict__ lse,
                                        const int32_t* __restrict__ lists, const int32_t* __restrict__ kv_len,
                                        const float* __restrict__ means, uint32_t* __restrict__ bits,
                                        const View<T>& gq, float* __restrict__ rows, const AttnArgs& a)
{
    using M = GqLds<T, D>;
    typedef typename Mma<T>::v8 v8;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = lane_id(), hi = lane >> 5;
    const int64_t id = xcd_contiguous(blockIdx.x, gridDim.x);
    const int bh = (int)(id / a.groups), g = (int)(id - bh * a.groups);
    const int b = bh / a.heads_q, h = bh - b * a.heads_q, hk = h / (a.heads_q / a.heads_k);
    const int tokens_q = (int)a.tokens_q, len = (int)seq_len(kv_len, b, a.tokens_k), past = len - tokens_q;
    const int i0 = g * QG, i = i0 + wave * 32 + (lane & 31), ic = i < tokens_q ? i : tokens_q - 1;
    // keys the lane's query and the group's last and first query see
    const int end = i0 + QG < tokens_q ? i0 + QG : tokens_q;
    const int mine = a.causal && past + i + 1 < len ? past + i + 1 : len;
    const int most = a.causal && past + end < len ? past + end : len;
    const int least = a.causal && past + i0 + 1 < len ? past + i0 + 1 : len;
    const float c = a.scale * LOG2E;
    const T* kb = k.at(b, 0, hk);
    const T* vb = v.at(b, 0, hk);
    const TileLoad<T, D, 4> load_k(k.st), load_v(v.st);
    const int visible = most > 0 ? (most + KB - 1) / KB : 0;
    ListWalk walk(lists + id * a.top, a.top, visible);
    // the group's bit at each of its blocks, for the other pass
    if (wave == 0) {
        ListWalk all(walk);
        do {
            if (all.left >> lane & 1) atomicOr(&bits[(bh * a.blocks + all.ids) * ((a.groups + 31) / 32) + g / 32], 1u << (g & 31));
        } while (all.more());
    }
    int blk = walk.next();
    if (blk >= 0) {
        load_k((T*)lds, kb, (int64_t)blk * KB, len - 1, wave);
        load_v((T*)(lds + M::TILE), vb, (int64_t)blk * KB, len - 1, wave);
    }
    v8 qf[D / 16], gf[D / 16];
    load_cols<T, D>(q.at(b, ic, h), qf);
    load_cols<T, D>(go.at(b, ic, h), gf);
    float dl = 0.f;
    {
        v8 of[D / 16];
        load_cols<T, D>(out.at(b, ic, h), of);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) dl = fmaf((float)gf[s][e], (float)of[s][e], dl);
        dl += __shfl_xor(dl, 32);
    }
    // a query that saw nothing has lse = -inf: P = exp2(S - inf) = 0; so has
    // one past the end, for the pass over the keys
    float nl = lse[(int64_t)bh * tokens_q + ic];
    nl = nl == -INFINITY || i >= tokens_q ? -INFINITY : -nl * LOG2E;
    acc16 acc[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t) acc[t] = zero16();
    float whole = 0.f, total = 0.f;              // sums of dS, as it is and rounded (R)
    float weight = 0.f, mean[D / 64] = {};  // of c, and c's dimensions lane, lane + 64
    const float* block_means = means + ((int64_t)b * a.heads_k + hk) * a.blocks * D;
    LaneAddresses<T, D> at(lds_address(lds), 0);
    auto step = [&](int stage, auto masked) __attribute__((always_inline)) {
        const int next = walk.next();
        wait_loads();
        __syncthreads();
        float mu[D / 64];  // before the loads to LDS, which it would else wait for
#pragma unroll
        for (int x = 0; x < D / 64; ++x) mu[x] = (block_means + (int64_t)blk * D)[lane + 64 * x];
        if (next >= 0) {
            char* to = lds + (stage ^ 1) * M::STAGE;
            load_k((T*)to, kb, (int64_t)next * KB, len - 1, wave);
            load_v((T*)(to + M::TILE), vb, (int64_t)next * KB, len - 1, wave);
        }
        float part = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            acc16 s = zero16(), p = zero16();
            constexpr uint32_t HALF = 32 * D * sizeof(T), STEP = 16 * D * sizeof(T);
            __builtin_amdgcn_sched_barrier(0);  // keeps the parts' registers apart
#pragma unroll
            for (int x = 0; x < D / 16; ++x) s = Mma<T>::mma(at.rows(x, t * HALF), qf[x], s);
#pragma unroll
            for (int x = 0; x < D / 16; ++x) p = Mma<T>::mma(at.rows(x, M::TILE + t * HALF), gf[x], p);
            interleave<D / 8, D / 8, 4>();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = exp2_fast(fmaf(s[r], c, nl));
            if constexpr (decltype(masked)::value) {
                const int upto = mine - blk * KB - 4 * hi - t * 32;  // against constants: no registers for the rows
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = c_row(r, 0) < upto ? s[r] : 0.f;
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                if (t == 0) part += s[r];
                s[r] *= p[r] - dl;
                whole += s[r];
            }
            const v8 ds0 = as_operand<T>(s, 0), ds1 = as_operand<T>(s, 1);
            total = add8(ds1, add8(ds0, total));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int y = 0; y < D / 32; ++y)
                    acc[y] = Mma<T>::mma(at.cols(y, t * HALF + x * STEP), x ? ds1 : ds0, acc[y]);
            interleave<D / 8, D / 16, 8>();
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (decltype(masked)::value) {
                // what rounding left, as a second operand
#pragma unroll
                for (int r = 0; r < 8; ++r) s[r] -= (float)ds0[r], s[8 + r] -= (float)ds1[r];
                const v8 rest0 = as_operand<T>(s, 0), rest1 = as_operand<T>(s, 1);
                total = add8(rest1, add8(rest0, total));
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < D / 32; ++y)
                        acc[y] = Mma<T>::mma(at.cols(y, t * HALF + x * STEP), x ? rest1 : rest0, acc[y]);
                interleave<D / 8, D / 16, 8>();
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        part = wave_sum(part);
        part = part < INFINITY ? part : 0.f;  // a NaN row must not reach its neighbours through c
        weight += part;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) mean[x] = fmaf(part, mu[x], mean[x]);
        at.move(stage ? (uint32_t)-1 * M::STAGE : M::STAGE);
        blk = next;
    };
    walk_blocks(step, [&] { return blk >= 0; }, [&] { return blk * KB + KB > least; });
    total += __shfl_xor(total, 32);
    whole += __shfl_xor(whole, 32);
    if (hi == 0) {
        float* row = rows + id * 2 * QG + wave * 32 + lane;
        row[0] = nl;
        row[QG] = dl + whole;
    }
    // c to LDS and back, to the lanes that hold its dimensions (of this wave only)
    float* cs = (float*)(lds + M::MEAN) + wave * D;
    const float inv = weight > 0.f ? 1.f / weight : 0.f;
#pragma unroll
    for (int x = 0; x < D / 64; ++x) cs[lane + 64 * x] = mean[x] * inv;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (i >= tokens_q) return;
    T* o = gq.at(b, i, h);
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float4v x = *(const float4v*)(cs + t * 32 + r * 8 + hi * 4) * total;
            store4<T>(o + t * 32 + r * 8 + hi * 4, (acc[t][4 * r] - x[0]) * a.scale, (acc[t][4 * r + 1] - x[1]) * a.scale,
                      (acc[t][4 * r + 2] - x[2]) * a.scale, (acc[t][4 * r + 3] - x[3]) * a.scale);
        }
}

template <typename T, int D>
__global__ __launch_bounds__(ATT_THREADS, 2) void k_attn_gq(View<const T> go, View<const T> q, View<const T> k,
                                                            View<const T> v, View<const T> out, const float* lse,
                                                            const int32_t* lists, const int32_t* kv_len,
                                                            const float* means, uint32_t* bits, View<T> gq,
                                                            float* rows, const AttnArgs a)
{
    __shared__ __align__(16) char s_lds[GqLds<T, D>::BYTES];
    attn_gq<T, D>(s_lds, go, q, k, v, out, lse, lists, kv_len, means, bits, gq, rows, a);
}

// Walks the (head of the key head, group of queries) pairs that list a block;
// every wave steps the same way. 64 words of the bit matrix are held by the
// lanes: a step costs a few scalar instructions instead of a dependent load.
struct Walk {
    const uint32_t* bits;  // of the first head, this block
    int64_t head_stride;
    int words, total;
    // state; lane l holds word base + l, its head and its first query (divided
    // there, once per 64 words, instead of per step)
    int base;
    uint64_t some;  // lanes with words left
    uint32_t held, left;
    int held_h, held_q, h, word_q, q0;
    __device__ __forceinline__ Walk(const uint32_t* p, int64_t stride, int n, int heads)
        : bits(p), head_stride(stride), words(n), total(n * heads), base(-64), some(0), held(0), left(0), held_h(0), held_q(0),
          h(0), word_q(0), q0(0)
    {
    }
    __device__ __forceinline__ bool next()
    {
        while (left == 0) {
            while (some == 0) {
                base += 64;
                if (base >= total) return false;
                const int i = base + (int)lane_id();
                held_h = (uint32_t)i / (uint32_t)words;
                held_q = (i - held_h * words) * 32 * QG;
                held = i < total ? bits[held_h * head_stride + (i - held_h * words)] : 0;
                some = ballot(held != 0);
            }
            const int at = __builtin_ctzll(some);
            some &= some - 1;
            left = __builtin_amdgcn_readlane(held, at);
            h = __builtin_amdgcn_readlane(held_h, at);
            word_q = __builtin_amdgcn_readlane(held_q, at);
        }
        q0 = word_q + __builtin_ctz(left) * QG;
        left &= left - 1;
        return true;
    }
};

// Blocks of one key head by the number of groups that list them, most first:
// the grid takes them in this order, so that the launch does not end on a
// block that many groups list (with no more blocks than CUs all start at once
// and none is needed). A counting sort on min(groups, ORDER_CLASSES - 1).
// Ties may fall in any order: a block's result does not depend on its place.
constexpr int ORDER_CLASSES = 1024;

__global__ __launch_bounds__(ATT_THREADS) void k_block_order(const uint32_t* __restrict__ bits,
                                                             uint32_t* __restrict__ order, const AttnArgs a)
{
    __shared__ uint32_t s_start[ORDER_CLASSES], s_part[ATT_THREADS];
    const int64_t bh = blockIdx.x, words = (a.groups + 31) / 32;
    const int per = a.heads_q / a.heads_k;
    const int64_t first = bh / a.heads_k * a.heads_q + bh % a.heads_k * per;  // the first query head
    for (int i = threadIdx.x; i < ORDER_CLASSES; i += ATT_THREADS) s_start[i] = 0;
    __syncthreads();
    auto cls = [&](int64_t blk) {
        uint32_t n = 0;
        for (int h = 0; h < per; ++h)
            for (int64_t w = 0; w < words; ++w) n += __popc(bits[((first + h) * a.blocks + blk) * words + w]);
        return ORDER_CLASSES - 1 - (n < ORDER_CLASSES - 1 ? n : ORDER_CLASSES - 1);
    };
    for (int64_t i = threadIdx.x; i < a.blocks; i += ATT_THREADS) atomicAdd(&s_start[cls(i)], 1u);
    __syncthreads();
    // exclusive sums: four classes a thread
    constexpr int PER = ORDER_CLASSES / ATT_THREADS;
    uint32_t v[PER], sum = 0;
    for (int i = 0; i < PER; ++i) sum += v[i] = s_start[threadIdx.x * PER + i];
    s_part[threadIdx.x] = sum;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < (int)threadIdx.x; ++i) before += s_part[i];
    for (int i = 0; i < PER; ++i) {
        s_start[threadIdx.x * PER + i] = before;
        before += v[i];
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < a.blocks; i += ATT_THREADS) order[bh * a.blocks + atomicAdd(&s_start[cls(i)], 1u)] = (uint32_t)i;
}

// gk and gv of a block of 64 keys, 64 queries a step: eight waves, one of
// either kind on each SIMD.
//   Four form P and dS of a 32 x 32 tile each (keys 32 kh, queries 32 qh), with
//   queries as rows, so that a lane holds one key, and leave them in LDS as the
//   operands they are for, rounded to the inputs' type, which is what the matrix
//   unit multiplies (gk and gv 2.35e-3 of their norm off in bf16, 1.66e-3 of it
//   their own rounding): what lane l rounded, lane l reads.
//   Four take the step before: gv^T += gout^T P or gk^T += q^T dS of 32 keys.
// Registers decide the shape. One wave with both sums (128 registers at dim
// 128), k and v (64) and S, dP (32) needs 340 and leaves a SIMD with one wave,
// which multiplies or computes exponentials but hardly both (measured: vector
// instructions behind a matrix instruction of the same wave are not hidden, of
// another wave they are). Split this way both kinds fit 256, and one
// multiplies while the other computes. The first kind is the longer one, so
// the other issues all loads. Three stages of queries: one loading, one per
// kind.
// What bounds it: a step's chain of products, exponentials, operands and
// barrier, and what a block costs besides its steps (bits, first loads, filling
// and draining the three stages, with no second workgroup on the CU): with lists
// of 8, 16, 32 and 64 blocks 0.54, 0.92, 1.5 and 2.8 ms at the size above, 10 us
// of each workgroup's 45 at 32. Without the loads, the sums or the scores alone
// the pass takes 1.2, 1.2 and 1.15 of its 1.44 ms. Loads two steps ahead in a
// fourth stage (row values through registers) are no faster, nor are twice the
// score waves, one half a step behind the other (1.75 ms), nor workgroups that
// go on to their next block (1.75 ms: the bookkeeping in every step costs more
// than the drain).
constexpr int GKV_THREADS = 512;

// LDS of the workgroup, in bytes.
template <typename T, int D>
struct GkvLds {
    static constexpr uint32_t TILE = Tile<D>::ELEMS * sizeof(T);          // q or gout of 64 queries
    static constexpr uint32_t STAGE = 2 * TILE;                            // q, gout
    static constexpr uint32_t OPS = 3 * STAGE, OP = 1024;                  // an operand: 16 bytes a lane
    static constexpr uint32_t ARRAY = 8 * OP, BUFFER = 2 * ARRAY;          // [2 kh][2 qh][2 steps]; P, dS
    static constexpr uint32_t ROWS = OPS + 2 * BUFFER, ROW_STAGE = 2 * 64 * 4;  // -lse in base 2, D
    static constexpr uint32_t BYTES = ROWS + 3 * ROW_STAGE;
};

// The steps of a block, the same for every wave, and this wave's loads.
template <typename T, int D>
struct GkvSteps {
    using M = GkvLds<T, D>;
    char* lds;
    const View<const T>&q, &go;
    const float* rows;
    TileLoad<T, D, 4> load_q, load_g;
    Walk w;
    int64_t head0, groups;  // first query head of the batch entry; groups a head
    int h0, b, tokens_q, wave, q0, half;  // wave: of the four that load
    __device__ __forceinline__ GkvSteps(char* l, const View<const T>& q_, const View<const T>& go_, const float* r,
                                        const Walk& walk, int b_, int h, const AttnArgs& a, int wave_)
        : lds(l), q(q_), go(go_), rows(r), load_q(q_.st), load_g(go_.st), w(walk), head0((int64_t)b_ * a.heads_q),
          groups(a.groups), h0(h), b(b_), tokens_q((int)a.tokens_q), wave(wave_), q0(0), half(1)
    {
    }
    __device__ __forceinline__ bool next()
    {
        if (half == 0 && q0 + 64 < tokens_q) {
            half = 1;
            q0 += 64;
            return true;
        }
        if (!w.next()) return false;
        half = 0;
        q0 = w.q0;
        return true;
    }
    __device__ __forceinline__ void load(uint32_t stage) const
    {
        const int h = h0 + w.h;
        T* to = (T*)(lds + stage * M::STAGE);
        load_q(to, q.at(b, 0, h), q0, tokens_q - 1, wave);
        load_g(to + Tile<D>::ELEMS, go.at(b, 0, h), q0, tokens_q - 1, wave);
        if (wave < 2) {  // the row values as they are: through registers they would wait for every load before them
            const float* src = rows + (((head0 + h) * groups + q0 / QG) * 2 + wave) * QG + q0 % QG + lane_id();
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void*)src,
                (__attribute__((address_space(3))) void*)(lds + M::ROWS + stage * M::ROW_STAGE + wave * 256), 4, 0, 0);
        }
    }
};

// P and dS, tile by tile.
template <typename T, int D>
__device__ __forceinline__ void gkv_scores(GkvSteps<T, D>& steps, const View<const T>& k, const View<const T>& v, int blk,
                                           int hk, int len, const AttnArgs& a, int wave)
{
    using M = GkvLds<T, D>;
    typedef typename Mma<T>::v8 v8;
    const int lane = lane_id(), hi = lane >> 5, kh = wave & 1, qh = wave >> 1;
    const int past = len - (int)a.tokens_q;
    const int key = blk * KB + kh * 32 + (lane & 31);
    const float c = a.scale * LOG2E;
    v8 kf[D / 16], vf[D / 16];
    {
        // keys past the end hold anything: take a valid one, its P is masked
        const int last = len > 0 ? len - 1 : 0, kc = key < last ? key : last;
        load_cols<T, D>(k.at(steps.b, kc, hk), kf);
        load_cols<T, D>(v.at(steps.b, kc, hk), vf);
    }
    LaneAddresses<T, D> at(lds_address(steps.lds), qh * 32);
    uint32_t stage = 0, buffer = 0;
    while (steps.next()) {
        __syncthreads();
        float nl[16], dl[16];
        const float* row = (const float*)(steps.lds + M::ROWS + stage * M::ROW_STAGE) + qh * 32 + 4 * hi;
#pragma unroll
        for (int r = 0; r < 16; ++r) nl[r] = row[c_row(r, 0)];
#pragma unroll
        for (int r = 0; r < 16; ++r) dl[r] = row[64 + c_row(r, 0)];
        acc16 s = zero16(), p = zero16();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) s = Mma<T>::mma(at.rows(x, 0), kf[x], s);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) p = Mma<T>::mma(at.rows(x, M::TILE), vf[x], p);
        interleave<D / 8, D / 8, 4>();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = exp2_fast(fmaf(s[r], c, nl[r]));
        const int first = steps.q0 + qh * 32;
        if ((blk + 1) * KB > (a.causal && past + first + 1 < len ? past + first + 1 : len)) {
            asm volatile("");  // a branch, not selects in every step
            // rows from `from` on see this lane's key
            const int from = key >= len ? 64 : (a.causal ? key - past - first - 4 * hi : 0);
#pragma unroll
            for (int r = 0; r < 16; ++r) s[r] = c_row(r, 0) >= from ? s[r] : 0.f;
        }
        v8* op = (v8*)(steps.lds + M::OPS + buffer * M::BUFFER + (kh * 2 + qh) * 2 * M::OP) + lane;
        op[0] = as_operand<T>(s, 0);
        op[M::OP / 16] = as_operand<T>(s, 1);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] *= p[r] - dl[r];
        op[M::ARRAY / 16] = as_operand<T>(s, 0);
        op[(M::ARRAY + M::OP) / 16] = as_operand<T>(s, 1);
        at.move(stage == 2 ? (uint32_t)-2 * M::STAGE : M::STAGE);
        stage = stage == 2 ? 0 : stage + 1;
        buffer ^= 1;
    }
    __syncthreads();  // hands over the last step
}

// gv (FOR_V) or gk of 32 keys: the step before that of the other waves.
template <typename T, int D, bool FOR_V>
__device__ __forceinline__ void gkv_sums(GkvSteps<T, D>& steps, const View<T>& result, int blk, int hk, const AttnArgs& a,
                                         int kh)
{
    using M = GkvLds<T, D>;
    typedef typename Mma<T>::v8 v8;
    const int lane = lane_id(), hi = lane >> 5, key = blk * KB + kh * 32 + (lane & 31);
    acc16 acc[D / 32];
#pragma unroll
    for (int t = 0; t < D / 32; ++t) acc[t] = zero16();
    LaneAddresses<T, D> at(lds_address(steps.lds), 0);
    auto sum = [&](uint32_t buffer) __attribute__((always_inline)) {
        const v8* op = (const v8*)(steps.lds + M::OPS + buffer * M::BUFFER + (FOR_V ? 0 : M::ARRAY) + kh * 4 * M::OP) + lane;
        __builtin_amdgcn_sched_barrier(0);
        v8 b[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) b[x] = op[x * (M::OP / 16)];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < D / 32; ++y)
                acc[y] = Mma<T>::mma(at.cols(y, (FOR_V ? M::TILE : 0) + x * 16 * D * sizeof(T)), b[x], acc[y]);
        interleave<D / 4, D / 8, 8, 4>();
        __builtin_amdgcn_sched_barrier(0);
    };
    uint32_t stage = 0, buffer = 1;
    bool more = steps.next(), some = false;
    if (more) steps.load(0);
    while (more) {
        wait_loads();
        __syncthreads();
        const uint32_t after = stage == 2 ? 0 : stage + 1;
        more = steps.next();
        if (more) steps.load(after);
        if (some) {
            sum(buffer);
            at.move(stage == 0 ? (uint32_t)-2 * M::STAGE : M::STAGE);  // from stage - 1 to stage
        }
        some = true;
        stage = after;
        buffer ^= 1;
    }
    __syncthreads();
    if (some) sum(buffer);
    if (key >= a.tokens_k) return;
    const float f = FOR_V ? 1.f : a.scale;
    T* o = result.at(steps.b, key, hk);
#pragma unroll
    for (int t = 0; t < D / 32; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            store4<T>(o + t * 32 + r * 8 + hi * 4, acc[t][4 * r] * f, acc[t][4 * r + 1] * f, acc[t][4 * r + 2] * f,
                      acc[t][4 * r + 3] * f);
}

template <typename T, int D>
__device__ __forceinline__ void attn_gkv(char* lds, const View<const T>& go, const View<const T>& q, const View<const T>& k,
                                         const View<const T>& v, const float* __restrict__ rows,
                                         const uint32_t* __restrict__ bits, const uint32_t* __restrict__ order,
                                         const int32_t* __restrict__ kv_len, const View<T>& gk, const View<T>& gv,
                                         const AttnArgs& a)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t id = xcd_contiguous(blockIdx.x, gridDim.x);
    const int bh = (int)(id / a.blocks), blk = order ? (int)order[id] : (int)(id - (int64_t)bh * a.blocks);
    const int b = bh / a.heads_k, hk = bh - b * a.heads_k, per = a.heads_q / a.heads_k;
    const int len = (int)seq_len(kv_len, b, a.tokens_k);
    const int words = (int)((a.groups + 31) / 32);
    const Walk w(bits + (((int64_t)b * a.heads_q + hk * per) * a.blocks + blk) * words, a.blocks * words, words, per);
    GkvSteps<T, D> steps(lds, q, go, rows, w, b, hk * per, a, wave & 3);
    if (wave < 4)
        gkv_scores<T, D>(steps, k, v, blk, hk, len, a, wave);
    else if (wave < 6)
        gkv_sums<T, D, true>(steps, gv, blk, hk, a, wave & 1);
    else
        gkv_sums<T, D, false>(steps, gk, blk, hk, a, wave & 1);
}

template <typename T, int D>
__global__ __launch_bounds__(GKV_THREADS, 2) void k_attn_gkv(View<const T> go, View<const T> q, View<const T> k,
                                                             View<const T> v, const float* rows, const uint32_t* bits,
                                                             const uint32_t* order, const int32_t* kv_len, View<T> gk,
                                                             View<T> gv, const AttnArgs a)
{
    // dynamic: with a static array of the same size the compiler's order of the
    // reads costs 4 %
    extern __shared__ __align__(16) char s_lds[];
    attn_gkv<T, D>(s_lds, go, q, k, v, rows, bits, order, kv_len, gk, gv, a);
}

static int64_t bits_words(int64_t batch, int64_t groups, int64_t blocks, int32_t heads_q)
{
    return batch * heads_q * blocks * ((groups + 31) / 32);
}

template <typename T, int D>
static gs_status attn_bwd_launch(const gs_tokens* go, const gs_tokens* q, const gs_tokens* k, const gs_tokens* v,
                                 const gs_tokens* out, const float* lse, const int32_t* list, const int32_t* kv_len,
                                 const gs_tokens* gq, const gs_tokens* gk, const gs_tokens* gv, float* rows,
                                 float* means, uint32_t* bits, uint32_t* order, int64_t batch, const AttnArgs& a, hipStream_t s)
{
    const int64_t lists = batch * a.heads_q * a.groups, blocks = batch * a.heads_k * a.blocks;
    const int64_t words = bits_words(batch, a.groups, a.blocks, a.heads_q);
    if (blocks > 0) {
        hipLaunchKernelGGL((k_attn_prepare<T, D>), dim3(grid_for((uint64_t)blocks, ATT_THREADS / 64)), dim3(ATT_THREADS), 0,
                           s, view_of<const T>(k), kv_len, means, bits, words, blocks, a);
        GS_CHECK_LAUNCH();
    }
    if (lists > 0) {
        hipLaunchKernelGGL((k_attn_gq<T, D>), dim3((unsigned)lists), dim3(ATT_THREADS), 0, s, view_of<const T>(go),
                           view_of<const T>(q), view_of<const T>(k), view_of<const T>(v), view_of<const T>(out), lse, list,
                           kv_len, means, bits, view_of<T>(gq), rows, a);
        GS_CHECK_LAUNCH();
    }
    if (blocks > 0) {
        const bool ordered = blocks > 256 && words > 0;
        if (ordered) {
            hipLaunchKernelGGL(k_block_order, dim3((unsigned)(batch * a.heads_k)), dim3(ATT_THREADS), 0, s, bits, order, a);
            GS_CHECK_LAUNCH();
        }
        constexpr uint32_t lds = GkvLds<T, D>::BYTES;
        if (lds > 65536 && hipFuncSetAttribute((const void*)k_attn_gkv<T, D>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)lds) != hipSuccess)
            return GS_ERR_HIP;
        hipLaunchKernelGGL((k_attn_gkv<T, D>), dim3((unsigned)blocks), dim3(GKV_THREADS), lds, s, view_of<const T>(go),
                           view_of<const T>(q), view_of<const T>(k), view_of<const T>(v), rows, bits,
                           ordered ? order : nullptr, kv_len, view_of<T>(gk), view_of<T>(gv), a);
        GS_CHECK_LAUNCH();
    }
    return GS_OK;
}

static size_t row_bytes(int64_t batch, int64_t tokens_q, int32_t heads_q)
{
    return (size_t)(batch * heads_q * ((tokens_q + QG - 1) / QG)) * 2 * QG * 4;
}

}  // namespace gs

extern "C" {

size_t gs_block_attn_bwd_workspace_bytes(int64_t batch, int64_t tokens_q, int64_t tokens_k, int32_t heads_q,
                                         int32_t heads_k, int32_t dim)
{
    using namespace gs;
    if (attn_check(batch, tokens_q, tokens_k, heads_q, heads_k, dim, GS_BF16, 1, 1.f) != GS_OK) return 0;
    const int64_t groups = (tokens_q + QG - 1) / QG, blocks = (tokens_k + KB - 1) / KB;
    return row_bytes(batch, tokens_q, heads_q) +
           (size_t)(bits_words(batch, groups, blocks, heads_q) + batch * heads_k * blocks * (dim + 1)) * 4 + 16;
}

gs_status gs_block_attn_bwd(const gs_tokens* gout, const gs_tokens* q, const gs_tokens* k, const gs_tokens* v,
                            const gs_tokens* out, const float* lse, const int32_t* list, int64_t batch,
                            int64_t tokens_q, int64_t tokens_k, int32_t heads_q, int32_t heads_k, int32_t dim,
                            int32_t dtype, const int32_t* kv_len, int32_t causal, int32_t top, float sm_scale,
                            const gs_tokens* gq, const gs_tokens* gk, const gs_tokens* gv, void* ws, size_t ws_bytes,
                            void* stream)
{
    using namespace gs;
    if (!gout || !q || !k || !v || !out || !gq || !gk || !gv) return GS_ERR_INVALID_ARGUMENT;
    const gs_status st = attn_check(batch, tokens_q, tokens_k, heads_q, heads_k, dim, dtype, top, sm_scale);
    if (st != GS_OK) return st;
    const bool queries = batch > 0 && tokens_q > 0, keys = batch > 0 && tokens_k > 0;
    if (!queries && !keys) return GS_OK;
    const size_t need = gs_block_attn_bwd_workspace_bytes(batch, tokens_q, tokens_k, heads_q, heads_k, dim);
    if (!ws || ((uintptr_t)ws & 15) || ws_bytes < need) return GS_ERR_INVALID_ARGUMENT;
    if (queries && (!gout->data || !q->data || !out->data || !gq->data || !lse || !list)) return GS_ERR_INVALID_ARGUMENT;
    if (keys && (!k->data || !v->data || !gk->data || !gv->data)) return GS_ERR_INVALID_ARGUMENT;
    if (queries)
        for (const gs_tokens* t : {gout, q, out, gq})
            if (!attn_view_ok(t, batch, tokens_q, heads_q)) return GS_ERR_UNSUPPORTED;
    if (keys)
        for (const gs_tokens* t : {k, v, gk, gv})
            if (!attn_view_ok(t, batch, tokens_k, heads_k)) return GS_ERR_UNSUPPORTED;
    const AttnArgs a{tokens_q, tokens_k, (tokens_q + QG - 1) / QG, (tokens_k + KB - 1) / KB, heads_q, heads_k,
                     causal != 0, top, 1, sm_scale};
    float* rows = (float*)ws;
    float* means = rows + row_bytes(batch, tokens_q, heads_q) / 4;
    uint32_t* bits = (uint32_t*)(means + batch * heads_k * a.blocks * dim);
    uint32_t* order = bits + bits_words(batch, a.groups, a.blocks, heads_q);
    const hipStream_t s = (hipStream_t)stream;
    if (dtype == GS_BF16)
        return dim == 128 ? attn_bwd_launch<bf16, 128>(gout, q, k, v, out, lse, list, kv_len, gq, gk, gv, rows, means, bits, order, batch, a, s)
                          : attn_bwd_launch<bf16, 64>(gout, q, k, v, out, lse, list, kv_len, gq, gk, gv, rows, means, bits, order, batch, a, s);
    return dim == 128 ? attn_bwd_launch<f16, 128>(gout, q, k, v, out, lse, list, kv_len, gq, gk, gv, rows, means, bits, order, batch, a, s)
                      : attn_bwd_launch<f16, 64>(gout, q, k, v, out, lse, list, kv_len, gq, gk, gv, rows, means, bits, order, batch, a, s);
}

}  // extern "C"
