// Shared by the attention kernels (block_attn.hip, block_attn_bwd.hip): the
// matrix instruction, the LDS tiles and their reads.
//
// Matrix tile: v_mfma 32x32x16. Lane l holds of A: row l & 31, of B: column
// l & 31, eight consecutive k from 8 (l >> 5); of C: column l & 31, rows
// 8 (i >> 2) + 4 (l >> 5) + (i & 3) for registers i = 0..15.
//
// Scores are formed transposed where queries are the columns (S^T = K Q^T): a
// lane then holds 16 keys of one query, so softmax needs one exchange between
// the two lane halves and the rescaling of the output is one factor per lane.
// And C's rows of registers 8g..8g+7 are, as a set, the 16 k of one B operand:
// slot s of half hi stands for row 16 g + 8 (s >> 2) + 4 hi + (s & 3). The
// order of k inside a product is free as long as A uses the same one, so
// probabilities go from C to B without crossing lanes, and A (the transposed
// values) is read from LDS in that order by two 4-row transposing reads.
#pragma once

#include <type_traits>

#include "tokens.h"

namespace gs {

constexpr int QG = GS_QUERY_GROUP, KB = GS_KEY_BLOCK;
constexpr int ATT_THREADS = 256;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

typedef float acc16 __attribute__((ext_vector_type(16)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef float float4v __attribute__((ext_vector_type(4)));

template <typename T>
struct Mma;
template <>
struct Mma<bf16> {
    typedef bf16 v8 __attribute__((ext_vector_type(8)));
    typedef bf16 v4 __attribute__((ext_vector_type(4)));
    static __device__ __forceinline__ acc16 mma(v8 a, v8 b, acc16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mma<f16> {
    typedef f16 v8 __attribute__((ext_vector_type(8)));
    typedef f16 v4 __attribute__((ext_vector_type(4)));
    static __device__ __forceinline__ acc16 mma(v8 a, v8 b, acc16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// A tile of 64 rows of D elements in LDS, in 16-byte chunks; chunk c of a row
// sits at c ^ swizzle(row). The swizzle serves both reads without bank
// conflicts (64 banks of 4 bytes): 16 lanes reading the same chunk of 16
// consecutive rows fall on 16 different 16-byte bank groups, and the four
// rows of a transposing read (rows 4m..4m+3, 64 bytes of each) on four
// different 64-byte ones.
template <int D>
struct Tile {
    static constexpr int CHUNKS = D / 8;
    static constexpr int ELEMS = KB * D;
    static __device__ __forceinline__ int swizzle(int row)
    {
        if constexpr (D == 128) return ((row & 3) << 2) | ((row >> 2) & 3);
        else return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
    }
    // element offset of chunk c of a row
    static __device__ __forceinline__ int at(int row, int c) { return (row * CHUNKS + (c ^ swizzle(row))) * 8; }
};

// Loads of 64 rows into a tile, straight to LDS (16 bytes a lane; the LDS side
// of such a load is linear in the lane, so the swizzle is applied to the
// global side). Each of WAVES waves issues CHUNKS / WAVES instructions; one
// covers 1024 bytes, ROWS rows. The lane's part of the address is a 32-bit
// offset formed once (its chunk differs between instructions by an XOR), the
// rest is uniform: one vector instruction per load.
template <typename T, int D, int WAVES>
struct TileLoad {
    static constexpr int CH = Tile<D>::CHUNKS, PER = CH / WAVES, ROWS = 64 / CH;
    uint32_t row, chunk;  // bytes
    int64_t stride;       // elements
    __device__ __forceinline__ explicit TileLoad(int64_t st) : stride(st)
    {
        const uint32_t r = lane_id() / CH, c = (lane_id() % CH) ^ Tile<D>::swizzle(r);
        row = r * (uint32_t)st * (uint32_t)sizeof(T);
        chunk = c * 16;
    }
    static __device__ __forceinline__ void one(T* tile, const void* src)
    {
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                         (__attribute__((address_space(3))) void*)tile, 16, 0, 0);
    }
    // Rows t0 .. t0 + 63; past `last`, row `last` again (masked by the reader,
    // but never a row that may hold anything).
    __device__ __forceinline__ void operator()(T* tile, const T* base, int64_t t0, int64_t last, int wave) const
    {
        const T* first = base + (t0 + wave * PER * ROWS) * stride;
        T* to = tile + wave * PER * 512;
        if (t0 + 63 <= last) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t x = D == 128 ? ((wave * PER + i) & 3) * 16 : ((wave * PER + i) & 1) * 32;
                one(to + i * 512, (const char*)(first + i * ROWS * stride) + ((chunk ^ x) + row));
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t x = D == 128 ? ((wave * PER + i) & 3) * 16 : ((wave * PER + i) & 1) * 32;
                const int64_t t = t0 + (wave * PER + i) * ROWS + lane_id() / CH;
                one(to + i * 512, (const char*)(base + (t < last ? t : last) * stride) + (chunk ^ x));
            }
        }
    }
};

// Order of the instructions around: READS LDS reads (and FIRST more before
// them) and MFMAS matrix instructions, the reads AHEAD of their use. (The
// compiler by itself reads one operand and waits for it.)
template <int READS, int MFMAS, int AHEAD, int FIRST = 0>
__device__ __forceinline__ void interleave()
{
    constexpr int PER = READS / MFMAS;
    static_assert(READS % MFMAS == 0 && AHEAD % PER == 0, "whole operands");
    __builtin_amdgcn_sched_group_barrier(0x100, FIRST + AHEAD, 0);
#pragma unroll
    for (int i = 0; i < MFMAS - AHEAD / PER; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, AHEAD / PER, 0);
}

// Loads to LDS are waited for here, before the barrier that hands the stage
// over. The compiler must not wait for them by itself, at reads of the other
// stage: it does so at the first transposing read unless the accesses carry
// alias scopes, which they get where the body is an inlined function with
// __restrict__ arguments. Hence each kernel below is one.
__device__ __forceinline__ void wait_loads()
{
    // vmcnt(0), the other counters as they are: a builtin, so that the compiler
    // knows that nothing is outstanding behind it
    __builtin_amdgcn_s_waitcnt(0x0f70);
    asm volatile("" ::: "memory");
}

// In both reads r0 is a multiple of 16, which the swizzle does not see: it goes
// into the instruction's offset, and the lane's address serves all of them.

// A operand, rows of the tile: row r0 + (l & 31), k = 16 step + 8 (l >> 5) ...
template <typename T, int D>
__device__ __forceinline__ typename Mma<T>::v8 read_rows(const T* tile, int r0, int step)
{
    const int l = lane_id();
    return *(const typename Mma<T>::v8*)(tile + r0 * D + Tile<D>::at(l & 31, step * 2 + (l >> 5)));
}

// A operand, columns of the tile as rows: row = column c0 + (l & 31), k = the
// tile's rows r0 + 8 (s >> 2) + 4 (l >> 5) + (s & 3) for slots s = 0..7.
// In each 16 lanes a transposing read takes 4 rows x 16 columns, 8 bytes a
// lane (lane i: row i / 4, columns 4 (i % 4) ...), and hands lane i column i.
template <typename T, int D>
__device__ __forceinline__ typename Mma<T>::v8 read_cols(const T* tile, int r0, int c0)
{
    const int l = lane_id(), hi = l >> 5, row = 4 * hi + ((l & 15) >> 2), col = c0 + (l & 16) + 4 * (l & 3);
    union {
        short4v h[2];
        typename Mma<T>::v8 v;
    } u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const T* p = tile + r0 * D + Tile<D>::at(8 * i + row, col >> 3) + (col & 7);
        u.h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v*)p);
    }
    return u.v;
}

// Address in LDS.
__device__ __forceinline__ uint32_t lds_address(const char* p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// The same reads with the lane's LDS addresses held in registers, of rows r0 ..
// of a tile that begins at `tile`: moving to another stage is one addition
// each, and the operand, the half and rows are offsets of the instruction.
template <typename T, int D>
struct LaneAddresses {
    uint32_t row[D / 16], col[D / 32][2];
    __device__ __forceinline__ LaneAddresses(uint32_t tile, uint32_t r0)
    {
        const int l = lane_id(), hi = l >> 5;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) row[x] = tile + (r0 * D + Tile<D>::at(l & 31, x * 2 + hi)) * sizeof(T);
#pragma unroll
        for (int y = 0; y < D / 32; ++y)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int c = y * 32 + (l & 16) + 4 * (l & 3);
                col[y][i] = tile + (r0 * D + Tile<D>::at(8 * i + 4 * hi + ((l & 15) >> 2), c >> 3) + (c & 7)) * sizeof(T);
            }
    }
    __device__ __forceinline__ void move(uint32_t by)
    {
#pragma unroll
        for (int x = 0; x < D / 16; ++x) row[x] += by;
#pragma unroll
        for (int y = 0; y < D / 32; ++y) col[y][0] += by, col[y][1] += by;
    }
    __device__ __forceinline__ typename Mma<T>::v8 rows(int x, uint32_t offset) const
    {
        return *(const __attribute__((address_space(3))) typename Mma<T>::v8*)(row[x] + offset);
    }
    __device__ __forceinline__ typename Mma<T>::v8 cols(int y, uint32_t offset) const
    {
        union {
            short4v h[2];
            typename Mma<T>::v8 v;
        } u;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            u.h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4v*)(col[y][i] + offset));
        return u.v;
    }
};

// B operand kept in registers: column = token, k = 16 step + 8 (l >> 5) ...
template <typename T, int D>
__device__ __forceinline__ void load_cols(const T* row, typename Mma<T>::v8 (&out)[D / 16])
{
    const int hi = lane_id() >> 5;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) out[s] = *(const typename Mma<T>::v8*)(row + s * 16 + hi * 8);
}

// Registers 8g..8g+7 of C as a B operand, rounded to nearest even.
template <typename T>
__device__ __forceinline__ typename Mma<T>::v8 as_operand(const acc16& c, int g)
{
    typename Mma<T>::v8 v;
#pragma unroll
    for (int s = 0; s < 8; ++s) v[s] = (T)c[8 * g + s];
    return v;
}

// sum += the eight elements, two at a time (products with one).
__device__ __forceinline__ float add8(Mma<bf16>::v8 v, float sum)
{
    typedef bf16 v2 __attribute__((ext_vector_type(2)));
    const v2 one = {(bf16)1.f, (bf16)1.f};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const v2 x = {v[i], v[i + 1]};
        sum = __builtin_amdgcn_fdot2_f32_bf16(x, one, sum, false);
    }
    return sum;
}
__device__ __forceinline__ float add8(Mma<f16>::v8 v, float sum)
{
    typedef f16 v2 __attribute__((ext_vector_type(2)));
    const v2 one = {(f16)1.f, (f16)1.f};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const v2 x = {v[i], v[i + 1]};
        sum = __builtin_amdgcn_fdot2(x, one, sum, false);
    }
    return sum;
}

__device__ __forceinline__ acc16 zero16()
{
    acc16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}

// Row of C that register i of this lane holds.
__device__ __forceinline__ int c_row(int i, int hi) { return 8 * (i >> 2) + 4 * hi + (i & 3); }

struct AttnArgs {
    int64_t tokens_q, tokens_k, groups, blocks;
    int32_t heads_q, heads_k, causal, top, splits;
    float scale;  // of the scores
};

// Valid keys of a sequence.
__device__ __forceinline__ int64_t seq_len(const int32_t* kv_len, int64_t b, int64_t tokens)
{
    const int64_t n = kv_len ? kv_len[b] : tokens;
    return n < 0 ? 0 : (n > tokens ? tokens : n);
}

// Walks the entries of a list that count, those that exceed every entry before
// them and lie inside the visible blocks: so none counts twice, in either
// direction, whatever the list holds. 64 entries are held by the wave's lanes:
// a step costs a few scalar instructions instead of a dependent load. With
// `step` only the entries `first`, first + step, ... are walked.
struct ListWalk {
    const int32_t* list;
    int64_t visible;
    int top, base, ids, most, first, step;  // ids: lane l holds entry base + l; most: the largest before them
    uint64_t left;
    __device__ __forceinline__ ListWalk(const int32_t* l, int n, int64_t vis, int from = 0, int by = 1)
        : list(l), visible(vis), top(n), base(0), most(-1), first(from), step(by)
    {
        fetch();
    }
    __device__ __forceinline__ void fetch()
    {
        const int j = base + (int)lane_id();
        ids = j < top ? list[j] : -1;
        const int before = j > 0 && j < top ? list[j - 1] : -1;
        const uint64_t up = ballot(ids > before);
        left = ballot(ids > max(before, most));
        if ((up & (up + 1)) == 0) {
            // as selected: rising entries, then none that rises, so the neighbour is the largest before
            if (up) most = max(most, __builtin_amdgcn_readlane(ids, __popcll(up) - 1));
        } else {
            left = 0;
#pragma unroll 1
            for (int i = 0; i < 64; ++i) {
                const int id = __builtin_amdgcn_readlane(ids, i);
                if (id > most) most = id, left |= 1ull << i;
            }
        }
        left &= ballot(ids < visible && (step == 1 || j % step == first));
    }
    // The next 64 entries, if there are any.
    __device__ __forceinline__ bool more()
    {
        base += 64;
        if (base >= top) return false;
        fetch();
        return true;
    }
    // The next block, or -1.
    __device__ __forceinline__ int next()
    {
        while (left == 0)
            if (!more()) return -1;
        const int j = __builtin_ctzll(left);
        left &= left - 1;
        return __builtin_amdgcn_readlane(ids, j);
    }
};

// The entries of an ascending list: blocks that every query of the group sees
// whole come first, those that a sequence's end or the causal limit cuts come
// last. So the first loop has no masks (and, one step per stage, constant LDS
// addresses); the second has.
template <typename Step, typename More, typename Cut>
__device__ __forceinline__ void walk_blocks(Step&& step, More&& more, Cut&& cut)
{
    int stage = 0;
    for (; more() && !cut(); stage ^= 1) step(stage, std::false_type{});
    for (; more(); stage ^= 1) step(stage, std::true_type{});
}

// 4 consecutive elements, 8 bytes.
template <typename T>
__device__ __forceinline__ void store4(T* p, float a, float b, float c, float d)
{
    typename Mma<T>::v4 v;
    v[0] = (T)a, v[1] = (T)b, v[2] = (T)c, v[3] = (T)d;
    *(typename Mma<T>::v4*)p = v;
}

// Host: the checks of sizes that both directions share.
gs_status attn_check(int64_t batch, int64_t tokens_q, int64_t tokens_k, int32_t heads_q, int32_t heads_k, int32_t dim,
                     int32_t dtype, int32_t top, float sm_scale);

// Rows on 16 bytes, and eight of them within the loads' 32-bit offsets.
inline bool attn_view_ok(const gs_tokens* t, int64_t batch, int64_t tokens, int64_t heads)
{
    return rows_aligned(t, batch, tokens, heads, 2, 16) && (tokens <= 1 || (t->stride_t >= 0 && t->stride_t < (1 << 27)));
}

}  // namespace gs
