// Matrix products by tiles, shared by the gated feed-forward block
// (gated_ff.hip) and the 4-bit linear layers (fp4.hip).
//
// A workgroup forms BM x BN elements of C = A B^T. Both operands pass through
// LDS in stages of KB bytes of a row's k (32 bytes a matrix step), loaded
// straight from memory into the stage that was read out last. A step's operands
// are read into registers while the step before it is on the matrix unit, also
// from one stage to the next: the one barrier per stage stands before its last
// step, whose operands are in registers by then. Behind it the next stage is whole
// and this one is free. A stage's loads are spread over the steps that follow:
// issued at once they fill the CU's one address path, and every wave behind it
// waits with its matrix instructions.
//
// Matrix tile: 32 x 32, 32 bytes of k a step. Lane l holds 16 bytes of k, half
// l >> 5, of row l & 31 of either operand. B goes first into the instruction, so
// that of C a lane holds row l & 31, columns 8 (i >> 2) + 4 (l >> 5) + (i & 3)
// for registers i = 0..15: four neighbours at a time.
//
// 4-bit elements take 8 to the place of two 16-bit ones: sizes of k below are in
// units of 2 bytes. A step then covers 64 of them, and a lane's 16 bytes are one
// block of 32 with its scale; the lane halves take the blocks of a stage in the
// order (2 hi + step), so that a lane's scales of all its steps are neighbours.
//
// An operand lies in memory either along k (its rows' k contiguous) or across
// it (TR: [k][rows], as the transposed matrices of a backward pass do); then
// its 16-bit elements are turned on the way from LDS to registers.
#pragma once

#include "block_attn.h"

namespace gs {

// The 16 x 16 x 32 product: of A row, of B column l & 15, eight k from 8 (l >> 4);
// of C column l & 15, rows 4 (l >> 4) on.
template <typename T>
__device__ __forceinline__ float4v mma16(typename Mma<T>::v8 a, typename Mma<T>::v8 b, float4v c)
{
    if constexpr (std::is_same<T, bf16>::value) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Two values of 4 bits a byte, of either operand of a scaled product.
struct fp4 {};
template <>
struct Mma<fp4> {
    typedef int v8 __attribute__((ext_vector_type(4)));
    typedef int v8i __attribute__((ext_vector_type(8)));
    // Scales: byte `s`, 0 or 1, of sa and sb, as exponents off 127.
    static __device__ __forceinline__ acc16 mma(v8 a, v8 b, acc16 c, int s, int sa, int sb)
    {
        const v8i x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
        return s == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb)
                      : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, 1, sa, 1, sb);
    }
};

// One operand's tile of ROWS rows in LDS, in chunks of 16 bytes, swizzled so
// that a wave's reads do not share banks (64 of 4 bytes).
//   along k:  [ROWS][KB]; chunk c of row r sits at c ^ f(r). 16 consecutive
//             rows, the same chunk of each: every chunk of 256 bytes once.
//   across:   [KB / 2][2 ROWS]; a turning read takes 4 rows of k, 64 bytes of
//             each: every 64 bytes of 256 once.
template <int ROWS, int KB, bool TR>
struct Panel {
    static constexpr int BYTES = ROWS * KB;
    static constexpr int PITCH = TR ? ROWS * 2 : KB, CHUNKS = PITCH / 16;
    static __device__ __forceinline__ int swizzle(int r)
    {
        if constexpr (!TR) return KB == 32 ? (r >> 3) & 1 : (KB == 64 ? (r >> 2) & 3 : (r >> 1) & 7);
        else if constexpr (ROWS >= 128) return ((r & 3) << 2) | ((r >> 2) & 3);
        else return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
    }
};

constexpr uint32_t PAST = 0x80000000u;  // an offset past every buffer: such loads give zeros

// `bytes` from p on, as the loads take it.
typedef uint32_t Buffer __attribute__((ext_vector_type(4)));
__device__ __forceinline__ Buffer buffer_of(const char* p, uint32_t bytes)
{
    const uint64_t at = (uint64_t)p;
    return Buffer{(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, bytes, 0x00027000u};
}

// 16 bytes a lane from a buffer, at a lane's offset and a uniform one that is
// inside the buffer, straight to LDS, lane after lane. In assembly
// because the compiler, which would have to keep these apart from reads of other
// stages, waits for all of them at a read where it cannot (two products in one
// kernel). They are waited for, and kept from reads, by `ready` below alone.
// M0 and a buffer from vector instructions need the wait states in between.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // that M0, which no code keeps over these, is clobbered
__device__ __forceinline__ void load_lds(Buffer src, uint32_t offset, uint32_t further, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(offset), "s"(src),
                 "s"(further)
                 : "memory", "m0");
}
__device__ __forceinline__ void load_lds_4(Buffer src, uint32_t offset, uint32_t lds)  // 4 bytes a lane
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(offset), "s"(src)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// Loads of a panel: WAVES waves, 16 bytes a lane, 1024 an instruction. The LDS
// side of such a load is linear in the lane, so the swizzle is on the memory side.
// With PAIR the panel's rows are of two matrices, PAIR of one and as many of the
// other in turn, and a wave loads of one of them.
template <int ROWS, int KB, bool TR, int WAVES, int PAIR = 0>
struct PanelLoad {
    using P = Panel<ROWS, KB, TR>;
    static constexpr int PER = P::BYTES / 1024 / WAVES, RPI = 1024 / P::PITCH;
    static_assert(PER * WAVES * 1024 == P::BYTES && RPI >= 1, "whole instructions");
    static_assert(!PAIR || (!TR && PAIR % (ROWS / WAVES) == 0), "a wave loads of one matrix");
    static constexpr int HALF = PAIR ? PAIR : 1;
    uint32_t off[PER];
    int wave;
    static __device__ __forceinline__ int row_of(int wave, int i) { return (wave * PER + i) * RPI + (int)lane_id() / P::CHUNKS; }
    static __device__ __forceinline__ int chunk_of(int row) { return ((int)lane_id() % P::CHUNKS) ^ P::swizzle(row); }
    // Which matrix of a pair the wave loads.
    static __device__ __forceinline__ int second(int wave) { return wave * (ROWS / WAVES) / HALF & 1; }
    __device__ __forceinline__ PanelLoad(uint32_t ld, int w) : wave(w)
    {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int r = row_of(w, i), m = PAIR ? r / (2 * HALF) * HALF + r % HALF : r;
            off[i] = (uint32_t)m * ld + chunk_of(r) * 16;
        }
    }
    // Load i of a stage from what is left of the matrix, `k` bytes of them of the
    // rows' own (behind the last stage of k a row goes on with what is not).
    __device__ __forceinline__ void one(Buffer src, uint32_t further, uint32_t lds, int i, int k) const
    {
        static_assert(TR || KB == 64 || PER % 2 == 0, "a load's chunk goes by whether it is odd");
        const int chunk = chunk_of(row_of(wave, KB == 64 ? 0 : i & 1));
        load_lds(src, TR || chunk * 16 < k ? off[i] : PAST, further, lds + (wave * PER + i) * 1024);
    }
};

// A lane's reads of 32 rows of a panel for one step: rows r0 + 32 t ..., where
// r0 is the wave's first row.
template <typename T, int ROWS, int KB, bool TR, int TILES>
struct PanelRead {
    using P = Panel<ROWS, KB, TR>;
    using V = typename Mma<T>::v8;
    static constexpr int STEPS = KB / 32, AT = TR ? 2 * TILES : STEPS;
    uint32_t at[AT];
    __device__ __forceinline__ explicit PanelRead(int r0)
    {
        const int l = lane_id(), hi = l >> 5;
        if constexpr (!TR) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int c = std::is_same<T, fp4>::value ? STEPS * hi + s : 2 * s + hi;
                at[s] = (r0 + (l & 31)) * KB + (c ^ P::swizzle(l & 31)) * 16;
            }
        } else {
            // slots 0..3 and 4..7 of a lane's k are rows 8 hi and 8 hi + 4 on, as an operand along k has them
#pragma unroll
            for (int t = 0; t < TILES; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int row = 8 * hi + 4 * i + ((l & 15) >> 2), c = r0 + 32 * t + (l & 16) + 4 * (l & 3);
                    at[2 * t + i] = row * P::PITCH + ((c >> 3) ^ P::swizzle(row)) * 16 + (c & 7) * 2;
                }
        }
    }
    __device__ __forceinline__ V operator()(const char* panel, int t, int s) const
    {
        if constexpr (!TR) {
            return *(const V*)(panel + at[s] + t * 32 * KB);
        } else {
            union {
                short4v h[2];
                V v;
            } u;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                u.h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) short4v*)(panel + at[2 * t + i] + s * 16 * P::PITCH));
            return u.v;
        }
    }
};

// An operand as the host describes it. Along k: row r, element k at data +
// r ld + k; across: data + k ld + r. A second matrix follows the first one along
// k (segments of k elements each), or is the other one of a pair.
struct Operand {
    const char* data[2];
    int64_t ld[2];  // bytes
    int64_t rows;   // of one matrix
};

// BM x BN elements by WM x WN waves. KG groups of such waves, each with stages of
// its own, share the sum over k; their sums meet in LDS, in order, in the first.
template <int BM_, int BN_, int WM_, int WN_, int KB_, int STAGES_, int KG_ = 1>
struct TileShape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, KB = KB_, STAGES = STAGES_, KG = KG_;
    static constexpr int WAVES = WM * WN, THREADS = WAVES * KG * 64, MT = BM / WM / 32, NT = BN / WN / 32;
    static constexpr int PER_SIMD = (THREADS / 64 + 3) / 4;  // waves that share a SIMD's registers
};

// The stages a workgroup walks: [first, last) of all segments' stages.
struct Walk {
    int64_t k;   // elements of a segment
    int stages;  // of a segment
    int first, last;
};

template <typename T, typename S, bool ATR, bool BTR, bool PAIR, bool TWO = false>
struct TileProduct {
    static constexpr int KE = S::KB / 2;  // elements of a stage
    using LoadA = PanelLoad<S::BM, S::KB, ATR, S::WAVES>;
    using LoadB = PanelLoad<S::BN, S::KB, BTR, S::WAVES, PAIR ? S::BN / S::WN / 2 : 0>;
    static constexpr int A_BYTES = LoadA::P::BYTES, STAGE = A_BYTES + LoadB::P::BYTES, GROUP = STAGE * S::STAGES;
    static constexpr bool FOUR = std::is_same<T, fp4>::value;
    static constexpr int LDS = GROUP * S::KG + (FOUR ? 3 * (S::BM + S::BN) * 16 : 0);
    // at the end: the other groups' sums, and below them a scratch for each wave of the first
    static constexpr int SUMS = S::MT * S::NT * 4096, FREE = GROUP * S::KG - (S::KG - 1) * S::WAVES * SUMS, SCRATCH = FREE / S::WAVES / 16 * 16;
    static constexpr int PANEL_LOADS = LoadA::PER + LoadB::PER, LOADS = PANEL_LOADS + FOUR;

    // An operand from the next stage on. Along k the buffer stays, and an offset
    // goes on (a row's own end is kept by `one`, that of the rows by the buffer);
    // across, rows of k pass, and their address goes on, past 32 bits, with the
    // bytes that are left.
    template <bool TR>
    struct Feed {
        Buffer src;
        const char* p;
        int64_t bytes, step;
        uint32_t further;
        static __device__ __forceinline__ uint32_t limit(int64_t n) { return (uint32_t)(n >> 31) ? 0x7fffffffu : (uint32_t)n; }
        __device__ __forceinline__ void at(const Operand& o, int which, int64_t r0, int64_t k, int64_t k0)
        {
            const int64_t ld = o.ld[which];
            if (TR) {
                p = o.data[which] + k0 * ld + r0 * 2;
                bytes = (k - 1 - k0) * ld + (o.rows - r0) * 2;
                step = KE * ld;
                further = 0;
            } else {
                src = buffer_of(o.data[which] + r0 * ld, limit((o.rows - 1 - r0) * ld + k * 2));
                further = (uint32_t)k0 * 2;
            }
        }
        __device__ __forceinline__ Buffer buffer(bool any) const { return TR ? buffer_of(p, any ? limit(bytes) : 0u) : src; }
        __device__ __forceinline__ void next()
        {
            if (TR) p += step, bytes -= step;
            else further += KE * 2;
        }
    };

    // Scales of 4-bit operands: 4 bytes a stage and row, loaded 4 stages at a time
    // (16 bytes of each of 16 rows an instruction: a load of 4 bytes of each of 64
    // rows takes the address path four times as long), [rows of A, rows of B][4
    // stages] in a ring of three, a group ahead of its stages.
    static constexpr int SCALE_GROUP = (S::BM + S::BN) * 16, SCALE_LOADS = SCALE_GROUP / 256 / S::WAVES;
    struct Scales {
        static_assert(S::WAVES % 2 == 0 && S::BM == S::BN, "a wave loads of one operand");
        Buffer src;
        uint32_t off, rows16, lds;
        __device__ __forceinline__ Scales(const Operand& a, const Operand& b, int64_t m0, int64_t n0, int bytes_of_row,
                                          const char* at, int wave)
        {
            const int first = wave % (S::WAVES / 2) * SCALE_LOADS * 16;
            const bool second = wave >= S::WAVES / 2;
            const int64_t ld = second ? b.ld[1] : a.ld[1], r0 = second ? n0 : m0;
            const int64_t bytes = ((second ? b.rows : a.rows) - 1 - r0) * ld + bytes_of_row;
            src = buffer_of((second ? b.data[1] : a.data[1]) + r0 * ld, (uint32_t)(bytes >> 31) ? 0x7fffffffu : (uint32_t)bytes);
            off = (uint32_t)(first + lane_id() / 4) * (uint32_t)ld + lane_id() % 4 * 4;
            rows16 = 16 * (uint32_t)ld;
            lds = uniform(lds_address(at)) + wave * SCALE_LOADS * 256;
        }
        // Load i of group g's, into place `ring` of the three.
        __device__ __forceinline__ void load(uint32_t g, uint32_t ring, int i) const
        {
            load_lds_4(src, off + (i * rows16 + g * 16), lds + ring * SCALE_GROUP + i * 256);
        }
        // The two bytes of this lane half's of a stage's four.
        static __device__ __forceinline__ int half(uint32_t x) { return x >> (lane_id() >> 5) * 16; }
    };

    // The sums of the first group's waves.
    static __device__ __forceinline__ void run(char* all, const Operand& a, const Operand& b, int64_t m0,
                                               int64_t n0, Walk w, int group, int wave, acc16 (&acc)[S::MT][S::NT])
    {
        const int per = (w.last - w.first + S::KG - 1) / S::KG;
        char* lds = all + group * GROUP;
        w.first += group * per;
        w.last = min(w.last, w.first + per);
        static_assert(!FOUR || (S::KB == 64 && S::KG == 1 && S::STAGES == 4 && 4 % SCALE_LOADS == 0), "the ring of scales");
        // loads that may be out when a stage has to be there
        constexpr int STEPS = S::KB / 32, LATER = (S::STAGES - 2) * LOADS;
        // a step is MT groups of matrix instructions; loads go EACH to a group, from the last step's on
        constexpr int EACH = (LOADS + S::MT * STEPS - 1) / (S::MT * STEPS), FIRST = LOADS < EACH * S::MT ? LOADS : EACH * S::MT;
        static_assert(STEPS % 2 == 0 && (S::STAGES == 2 || S::STAGES == 4) && LATER + FIRST < 64, "steps in pairs; loads out fit the wait's field");
        const LoadA load_a((uint32_t)a.ld[0], wave);
        const int mine = PAIR ? LoadB::second(wave) : w.first >= w.stages;
        LoadB load_b((uint32_t)b.ld[mine], wave);
        const PanelRead<T, S::BM, S::KB, ATR, S::MT> read_a(wave / S::WN * (S::BM / S::WM));
        const PanelRead<T, S::BN, S::KB, BTR, S::NT> read_b(wave % S::WN * (S::BN / S::WN));
#pragma unroll
        for (int i = 0; i < S::MT; ++i)
#pragma unroll
            for (int j = 0; j < S::NT; ++j) acc[i][j] = zero16();
        int in = w.first - (w.first >= w.stages ? w.stages : 0);  // stage of its segment, the next to load
        int left = w.last - w.first, k = (int)(w.k - (int64_t)in * KE) * 2;
        Feed<ATR> fa;
        Feed<BTR> fb;
        fa.at(a, w.first >= w.stages, m0, w.k, (int64_t)in * KE);
        fb.at(b, mine, n0, w.k, (int64_t)in * KE);
        // of the stage whose loads are being issued: where from and where to
        Buffer from_a, from_b;
        uint32_t further_a, further_b, to;
        int k_of;
        auto prepare = [&](const char* stage) __attribute__((always_inline)) {
            const bool any = left > 0;
            from_a = fa.buffer(any);
            from_b = fb.buffer(any);
            further_a = any ? fa.further : 0;  // never past the buffer's size, from which it is taken off
            further_b = any ? fb.further : 0;
            k_of = any ? k : 0;
            to = uniform(lds_address(stage));
            --left, ++in, k -= KE * 2;
            fa.next();
            fb.next();
        };
        // with stage s goes load s % 4 of the scales of the four stages that follow the four of s
        const char* scales = all + GROUP * S::KG;
        const Scales scale(a, b, m0, n0, (int)(w.k + 31) / 32 * 4, scales, wave);
        uint32_t scale_group = 1, scale_ring = 1;
        int scale_part = 0;
        // the loads of group `g` behind the barrier
        auto load = [&](int g) __attribute__((always_inline)) {
#pragma unroll
            for (int i = g * EACH; i < (g + 1) * EACH && i < LOADS; ++i) {
                if (i < LoadA::PER) load_a.one(from_a, further_a, to, i, k_of);
                else if (i < PANEL_LOADS) load_b.one(from_b, further_b, to + A_BYTES, i - LoadA::PER, k_of);
                else if constexpr (FOUR) scale.load(scale_group, scale_ring, scale_part);
            }
        };
        // after a stage's last load: on to the second segment?
        auto turn = [&]() __attribute__((always_inline)) {
            if (TWO && in == w.stages && left > 0) {
                k = (int)w.k * 2;
                fa.at(a, 1, m0, w.k, 0);
                fb.at(b, 1, n0, w.k, 0);
                load_b = LoadB((uint32_t)b.ld[1], wave);
            }
        };
        // `out` loads may be left out; all LDS reads are done
        auto ready = [&](auto out) __attribute__((always_inline)) {
            constexpr int N = decltype(out)::value;
            __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | (N >> 4) << 14);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
        };
        typename Mma<T>::v8 ra[2][S::MT], rb[2][S::NT];
        // operand i of a step's: B's, then A's
        auto read = [&](const char* stage, int step, int to, int i) __attribute__((always_inline)) {
            if (i < S::NT) rb[to][i] = read_b(stage + A_BYTES, i, step);
            else ra[to][i - S::NT] = read_a(stage, i - S::NT, step);
        };
        constexpr int READS = S::NT + S::MT;
        int sa[S::MT], sb[S::NT];
        uint32_t next_sa[S::MT], next_sb[S::NT];
        auto multiply = [&](int step, int i) __attribute__((always_inline)) {
            const int from = step & 1;
#pragma unroll
            for (int j = 0; j < S::NT; ++j) {
                if constexpr (FOUR) acc[i][j] = Mma<T>::mma(rb[from][j], ra[from][i], acc[i][j], step, sb[j], sa[i]);
                else acc[i][j] = Mma<T>::mma(rb[from][j], ra[from][i], acc[i][j]);
            }
        };
        if constexpr (FOUR) {
#pragma unroll
            for (int i = 0; i < SCALE_LOADS; ++i) scale.load(0, 0, i);
        }
#pragma unroll
        for (int t = 0; t < S::STAGES; ++t) {
            prepare(lds + t * STAGE);
            scale_part = t % SCALE_LOADS;
#pragma unroll
            for (int g = 0; g < (t < S::STAGES - 1 ? S::MT * STEPS : S::MT); ++g) load(g);
            if (t < S::STAGES - 1) turn();
        }
        ready(std::integral_constant<int, (S::STAGES - 2) * LOADS + FIRST>{});
#pragma unroll
        for (int i = 0; i < READS; ++i) read(lds, 0, 0, i);
        // this lane's scales of a stage, all four bytes of each row: place `ring`, stage `slot` of its four
        const char* scale_rows = scales + (wave / S::WN * (S::BM / S::WM) + (lane_id() & 31)) * 16;
        const char* scale_cols = scales + (S::BM + wave % S::WN * (S::BN / S::WN) + (lane_id() & 31)) * 16;
        auto next_scales = [&](uint32_t ring, int slot) __attribute__((always_inline)) {
            const char *rows = scale_rows + ring * SCALE_GROUP, *cols = scale_cols + ring * SCALE_GROUP;
#pragma unroll
            for (int i = 0; i < S::MT; ++i) next_sa[i] = *(const uint32_t*)(rows + i * 512 + slot * 4);
#pragma unroll
            for (int j = 0; j < S::NT; ++j) next_sb[j] = *(const uint32_t*)(cols + j * 512 + slot * 4);
        };
        // of the last stage's four bytes only those of k's own blocks count
        const int last_blocks = (int)(w.k - (int64_t)(w.stages - 1) * KE) / 8;
        const uint32_t last_mask = last_blocks < 4 ? (1u << 8 * last_blocks) - 1 : ~0u;
        uint32_t ring = 0, ring_next = 1, pair = 0;  // places of the scales, and of the pair of stages among the ring's
        if constexpr (FOUR) next_scales(0, 0);
        int t = w.first;
        // One stage; `u`: its place in its pair.
        auto stage_of = [&](int u) __attribute__((always_inline)) {
            const char* here = lds + pair * 2 * STAGE;
            const char* stage = here + u * STAGE;
            const char* next = S::STAGES == 2 ? lds + (u ^ 1) * STAGE : (u == 0 ? here + STAGE : lds + (pair ^ 1) * 2 * STAGE);
            if constexpr (FOUR) {
                const uint32_t mask = t < w.stages - 1 ? ~0u : (t == w.stages - 1 ? last_mask : 0u);
#pragma unroll
                for (int i = 0; i < S::MT; ++i) sa[i] = Scales::half(next_sa[i] & mask);
#pragma unroll
                for (int j = 0; j < S::NT; ++j) sb[j] = Scales::half(next_sb[j] & mask);
            }
            // The order is kept as written: between two groups of matrix instructions go a few of the next
            // step's reads and a load. Of the last step, one group stands before the barrier.
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const bool last = s == STEPS - 1;
#pragma unroll
                for (int i = 0; i < S::MT; ++i) {
                    if (i == 0 && s > 0 && TWO && s == STEPS - 1) turn();
                    if (S::MT > 1) {
                        multiply(s, i);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    if (last && i == 0) {
                        ready(std::integral_constant<int, LATER>{});
                        prepare(stage);
                        if constexpr (FOUR) {
                            scale_part = (pair * 2 + u) % SCALE_LOADS;
                            if (u == 0 && pair == 0) ++scale_group, scale_ring = scale_ring == 2 ? 0 : scale_ring + 1;
                        }
                    }
                    // the reads before the last group, of which the last step has one fewer
                    constexpr int G = S::MT > 2 ? S::MT - 1 : S::MT;
                    const int parts = S::MT > 1 && last && G > 1 ? G - 1 : G, p = S::MT > 1 && last && G > 1 ? i - 1 : i;
#pragma unroll
                    for (int r = 0; r < READS; ++r)
                        if (p >= 0 && p < parts && r * parts / READS == p) read(last ? next : stage, last ? 0 : s + 1, (s + 1) & 1, r);
                    load(last ? i : (s + 1) * S::MT + i);
                    if (FOUR && s == 0 && i == S::MT - 1) {
                        if (u == 1 && pair == 1) ring = ring_next, ring_next = ring_next == 2 ? 0 : ring_next + 1;
                        next_scales(ring, u == 0 ? pair * 2 + 1 : (pair ^ 1) * 2);
                    }
                    if (S::MT > 1) __builtin_amdgcn_sched_barrier(0);
                    else multiply(s, i);
                }
            }
        };
        // two at a time, so that a stage's place is a constant; one past the end adds zeros
        for (int n = 0; n < per; n += 2) {
            stage_of(0);
            ++t;
            stage_of(1);
            ++t;
            if (S::STAGES > 2) pair ^= 1;
        }
        // what was loaded past the end has landed and all reads are done: LDS is free
        ready(std::integral_constant<int, 0>{});
        if constexpr (S::KG > 1) {
            float4v* at = (float4v*)(all + FREE + wave * SUMS) + lane_id();
            const auto each = [&](auto f) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < S::MT; ++i)
#pragma unroll
                    for (int j = 0; j < S::NT; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) f(acc[i][j], r, ((i * S::NT + j) * 4 + r) * 64);
            };
            if (group > 0)
                each([&](acc16& c, int r, int to) __attribute__((always_inline)) {
                    at[(group - 1) * S::WAVES * (SUMS / 16) + to] = float4v{c[4 * r], c[4 * r + 1], c[4 * r + 2], c[4 * r + 3]};
                });
            __syncthreads();
            if (group == 0) {
#pragma unroll
                for (int g = 0; g < S::KG - 1; ++g)
                    each([&](acc16& c, int r, int to) __attribute__((always_inline)) {
                        const float4v x = at[g * S::WAVES * (SUMS / 16) + to];
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[4 * r + e] += x[e];
                    });
            }
        }
    }
};

// A wave's scratch in LDS for 32 rows of W bytes (32, 64 or 128), in chunks of 16
// swizzled as a panel's: rows of C are written four columns at a time and leave
// as whole rows, 16 bytes a lane (without it a store would hold 16 bytes of each
// of 32 rows).
template <int W>
struct Rows {
    char* p;
    static __device__ __forceinline__ int at(int row, int byte)
    {
        return row * W + (((byte >> 4) ^ Panel<32, W, false>::swizzle(row)) << 4) + (byte & 15);
    }
    // This lane's row (l & 31), at a byte of it.
    template <typename V>
    __device__ __forceinline__ void put(int byte, const V& v) const
    {
        *(V*)(p + at(lane_id() & 31, byte)) = v;
    }
    template <typename V>
    __device__ __forceinline__ V get(int byte) const
    {
        return *(const V*)(p + at(lane_id() & 31, byte));
    }
    // Rows first .. rows - 1 to memory, V at a time, `bytes` of each (a multiple of V's).
    template <typename V>
    __device__ __forceinline__ void store_as(char* to, int64_t ld, int64_t rows, int64_t bytes, int64_t first) const
    {
        constexpr int N = W / sizeof(V);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
            const int row = (k * 64 + lane_id()) / N, byte = (lane_id() % N) * sizeof(V);
            const V v = *(const V*)(p + at(row, byte));
            if (row >= first && row < rows && byte < bytes) *(V*)(to + row * ld + byte) = v;
        }
    }
    __device__ __forceinline__ void store(char* to, int64_t ld, int64_t rows, int64_t bytes, int64_t first = 0) const
    {
        store_as<uint4>(to, ld, rows, bytes, first);
    }
    // The same from memory to registers, zeros past the end, and from those to the scratch.
    template <typename V, int K>
    static __device__ __forceinline__ void fetch(V (&v)[K], const char* from, int64_t ld, int64_t rows, int64_t bytes)
    {
        constexpr int N = W / sizeof(V);
        static_assert(K == N / 2, "a lane's part of 32 rows");
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int row = (k * 64 + lane_id()) / N, byte = (lane_id() % N) * sizeof(V);
            v[k] = V{};
            if (row < rows && byte < bytes) v[k] = *(const V*)(from + row * ld + byte);
        }
    }
    template <typename V, int K>
    __device__ __forceinline__ void put_all(const V (&v)[K]) const
    {
        constexpr int N = W / sizeof(V);
#pragma unroll
        for (int k = 0; k < K; ++k) *(V*)(p + at((k * 64 + lane_id()) / N, (lane_id() % N) * sizeof(V))) = v[k];
    }
    // Rows of a multiple of 8 bytes.
    __device__ __forceinline__ void store8(char* to, int64_t ld, int64_t rows, int64_t bytes) const
    {
        store_as<uint2>(to, ld, rows, bytes, 0);
    }
};

// Waits for this wave's LDS accesses (its lanes exchange values through a
// scratch of its own, without a barrier).
__device__ __forceinline__ void wait_lds()
{
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0), the other counters as they are
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// Workgroup -> tile: each XCD takes a contiguous range, in which 8 row tiles by
// all column tiles come first, so that what runs at once shares rows of both
// operands in its L2.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t mt, uint32_t nt, uint32_t& m, uint32_t& n)
{
    constexpr uint32_t GROUP = 8;
    const uint32_t g = id / (GROUP * nt), in = id - g * GROUP * nt;
    const uint32_t rows = min(mt - g * GROUP, GROUP);
    n = uniform(in / rows);
    m = uniform(g * GROUP + (in - n * rows));
}

}  // namespace gs
