// attention.hpp -- what the kernels of attention share: the matrix products of a
// wave, tiles of rows in LDS, and which keys a query sees.
//
// All products are 32 x 32 results of one wave with v_mfma_f32_32x32x16 (bf16,
// fp16) or eight v_mfma_f32_32x32x2 (fp32).  A lane's operands are eight
// consecutive numbers of k of one row (A) or column (B) lane % 32, the upper 32
// lanes those after the lower ones'; its results are 16 rows of column
// lane % 32, register i being row 8*(i / 4) + 4*(lane / 32) + i % 4.
//
// The kernels keep one side of every product in registers, a column a lane
// (queries in the forward pass and the gradient of q, keys in the gradients of k
// and v), and stream rows of the other side through LDS.  With scores as results
// (streamed row, own column), softmax statistics are a lane's own but for one
// exchange between the halves of the wave, and the weights P are at once the B
// operand of the product that follows: its k are the streamed rows, and any
// order of them does as long as both operands have the same.  Slot i of a
// 16-row step is row 8*(i / 4) + 4*(lane / 32) + i % 4 in both.  The A operand of
// that product is the tile read along its rows, transposed on the way by
// ds_read_b64_tr_b16.
//
// A tile's rows lie in LDS in chunks of 16 bytes that are exchanged within a row
// (chunk c of row r at place c ^ swizzle(r)), so that eight rows read along a
// column, and four rows read transposed, fall on all banks.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#define BASP_HD __host__ __device__
#include "attention_plan.hpp"
#include "barrier.hpp"
#include "rowvec.hpp"

namespace basp {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

template <typename T> struct Of;
template <> struct Of<__bf16> {
    typedef __bf16 x8 __attribute__((ext_vector_type(8)));
};
template <> struct Of<_Float16> {
    typedef _Float16 x8 __attribute__((ext_vector_type(8)));
};
template <> struct Of<float> {          // read at addresses of whole 16 bytes
    typedef float x8 __attribute__((ext_vector_type(8), aligned(16)));
};
template <typename T> using Vec8 = typename Of<T>::x8;

__device__ inline f32x16 product(Vec8<__bf16> a, Vec8<__bf16> b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ inline f32x16 product(Vec8<_Float16> a, Vec8<_Float16> b, f32x16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
// Each of the eight takes one number of k from either half of the wave.
__device__ inline f32x16 product(Vec8<float> a, Vec8<float> b, f32x16 c)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
    return c;
}

// Row of register i of a result, and of slot i of a 16-row step.
__device__ inline int row_of(int i, int half) { return 8 * (i / 4) + 4 * half + i % 4; }

// Registers 8*s to 8*s + 7 of a result as the B operand of the next product: the
// one rounding of P (or dS) to the inputs' type, which the matrix instruction
// takes.  The softmax's sum is taken of the unrounded values.
template <typename T>
__device__ inline Vec8<T> operand(const f32x16 &c, int s)
{
    Vec8<T> r;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        r[i] = static_cast<T>(c[8 * s + i]);
    return r;
}

// sum + 0 * (the numbers): NaN if one of them is infinite or NaN.
__device__ inline float zeros_of(Vec8<__bf16> x, float sum)
{
    typedef __bf16 x2 __attribute__((ext_vector_type(2)));
    const x2 zero = {};
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        sum = __builtin_amdgcn_fdot2_f32_bf16(x2{x[i], x[i + 1]}, zero, sum, false);
    return sum;
}
__device__ inline float zeros_of(Vec8<_Float16> x, float sum)
{
    typedef _Float16 x2 __attribute__((ext_vector_type(2)));
    const x2 zero = {};
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        sum = __builtin_amdgcn_fdot2(x2{x[i], x[i + 1]}, zero, sum, false);
    return sum;
}
__device__ inline float zeros_of(Vec8<float> x, float sum)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        sum = fmaf(x[i], 0.f, sum);
    return sum;
}

// The value of the lane across the wave.
__device__ inline float other_half(float x)
{
    const uint32_t w = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return __builtin_bit_cast(float, (threadIdx.x & 32) ? uint32_t(r[0]) : uint32_t(r[1]));
}

// ------------------------------------------------------------------- tiles --

typedef __attribute__((address_space(3))) char lds_char;

// The lane's number, of which the compiler does not know that it is the same in
// every step: addresses made of it are computed where they are used instead of
// being kept in registers.
__device__ inline uint32_t lane_here()
{
    uint32_t lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// The place of an LDS address in the work-group's share.
__device__ inline uint32_t lds_place(const void *p)
{
    return uint32_t(reinterpret_cast<uintptr_t>((lds_char *)const_cast<char *>(static_cast<const char *>(p))));
}

// `bytes` bytes of memory from an address that is the same for the wave: reads
// beyond them give zeros.
__device__ inline u32x4 memory_rows(const void *from, uint32_t bytes)
{
    const uint64_t at = reinterpret_cast<uint64_t>(from);
    return u32x4{scalar(uint32_t(at)), scalar(uint32_t(at >> 32)) & 0xffffu, scalar(bytes), 0x00020000u};
}

// BYTES bytes of each lane, `off` bytes into memory, straight to LDS, lane after
// lane from place `to` on (lds_place).  Written as an instruction, since the compiler would wait
// for it before the next transposed read of any part of LDS; it is complete after
// wait_tiles.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"         // m0 is named so that the compiler sets it anew for itself
template <int BYTES>
__device__ inline void copy_to_lds(uint32_t to, u32x4 from, uint32_t off)
{
    const uint32_t at = scalar(to);
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                     :: "s"(at), "v"(off), "s"(from) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                     :: "s"(at), "v"(off), "s"(from) : "memory", "m0");
}
#pragma clang diagnostic pop

// ROWS rows of C channels in LDS.
template <typename T, int C, int ROWS>
struct Tile {
    static constexpr int kRow = C * sizeof(T), kChunks = kRow / 16, kBytes = ROWS * kRow;
    static constexpr int kPer = 16 / sizeof(T);        // numbers of a chunk

    // Eight chunks a row: two rows span the banks, so that the row's lowest bit
    // is left out.  Sixteen and more: the low bits of the row move chunks by
    // four, the next ones by one.
    static __device__ inline uint32_t swizzle(uint32_t r)
    {
        return kChunks == 8 ? ((r >> 1 & 1) << 2) | (r >> 2 & 3) : ((r & 3) << 2) | (r >> 2 & 3);
    }

    // The A operand of scores: row `row0` + lane % 32, channels 16*s on.
    static __device__ inline Vec8<T> along_channels(const char *tile, int row0, int s, uint32_t lane = threadIdx.x & 63)
    {
        const uint32_t r = lane & 31, half = lane >> 5;
        const char *const at = tile + (row0 + r) * kRow;
        if constexpr (sizeof(T) == 2) {
            const uint32_t c = (2 * s) ^ (half ^ swizzle(r));
            return *reinterpret_cast<const Vec8<T> *>(at + c * 16);
        } else {
            typedef float x4 __attribute__((ext_vector_type(4)));
            const uint32_t c = (4 * s) ^ ((2 * half) ^ swizzle(r));
            const x4 lo = *reinterpret_cast<const x4 *>(at + c * 16), hi = *reinterpret_cast<const x4 *>(at + (c ^ 1) * 16);
            return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }

    // The A operand of sums over rows: channel 32*block + lane % 32 of the slots
    // of the 16 rows from row0 on.
    static __device__ inline Vec8<T> along_rows(const char *tile, int row0, int block, uint32_t lane = threadIdx.x & 63)
    {
        const uint32_t half = lane >> 5;
        if constexpr (sizeof(T) == 2) {
            // 16 lanes read four rows of 16 channels, four channels each, and
            // receive a channel each of the four rows
            const uint32_t l = lane & 15, r = 4 * half + (l >> 2), group = lane >> 4 & 1;
            const uint32_t c = (2 * group + (l >> 1 & 1)) ^ swizzle(r);
            typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
            s16x4 part[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // swizzle(r + 8 j) == swizzle(r) ^ 2 j
                const uint32_t off = (row0 + 8 * j + r) * kRow + ((4 * block) ^ (2 * j) ^ c) * 16 + (l & 1) * 8;
                part[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds_char *)(tile + off));
            }
            typedef short s16x8 __attribute__((ext_vector_type(8)));
            return __builtin_bit_cast(Vec8<T>, s16x8(__builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7)));
        } else {
            Vec8<T> v;
            const uint32_t c = block * 8 + ((lane & 31) >> 2);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t r = row0 + row_of(i, half);
                v[i] = *reinterpret_cast<const float *>(tile + r * kRow + ((c ^ swizzle(r)) * 16) + (lane & 3) * 4);
            }
            return v;
        }
    }

    // One number.
    static __device__ inline float at(const char *tile, int row, int channel)
    {
        const uint32_t c = (uint32_t(channel) / kPer) ^ swizzle(row);
        return static_cast<float>(*reinterpret_cast<const T *>(tile + row * kRow + c * 16 + (channel % kPer) * sizeof(T)));
    }

    // Brings rows of `d` channels, `token` bytes apart, into a tile by THREADS
    // threads, with zeros after the last row and channel d.  DIRECT: rows of whole
    // 16-byte chunks at 16-byte addresses go from memory to LDS without passing
    // registers; the loads are complete after wait_tiles and a barrier.
    //
    // place: lds_place(tile).  off: the places of a thread's chunks from the first
    // row, the same for every tile (load_offsets).
    template <int THREADS, int STEPS>
    static __device__ inline void load_offsets(uint32_t (&off)[STEPS], uint32_t token, int d)
    {
#pragma unroll
        for (int p = 0; p < STEPS; ++p) {
            const uint32_t i = p * THREADS + threadIdx.x % THREADS, r = i / kChunks, c = (i % kChunks) ^ swizzle(r);
            // beyond any buffer: reads as zeros
            off[p] = int(c) * kPer < d ? r * token + c * 16 : 0x80000000u;
        }
    }

    template <int THREADS, bool DIRECT, int STEPS>
    static __device__ inline void load(char *__restrict__ tile, uint32_t place, const uint32_t (&off)[STEPS], const char *from,
                                       uint32_t token, int rows, int d)
    {
        static_assert(kBytes == 16 * THREADS * STEPS, "whole rounds of the threads");
        if constexpr (DIRECT) {
            const uint32_t wave = scalar(threadIdx.x % THREADS >> 6);
            const u32x4 rows_of = memory_rows(from, rows * token);
#pragma unroll
            for (int p = 0; p < STEPS; ++p)
                copy_to_lds<16>(place + (p * THREADS + wave * 64) * 16, rows_of, off[p]);
        } else {
            // all on their way before the first is stored
            typedef T xn __attribute__((ext_vector_type(kPer)));
            xn x[STEPS];
#pragma unroll
            for (int p = 0; p < STEPS; ++p) {
                const int r = (p * THREADS + threadIdx.x % THREADS) / kChunks, c = (threadIdx.x % kChunks) ^ swizzle(r);
                x[p] = chunk(from + uint64_t(r < rows ? r : rows - 1) * token, c * kPer, d);        // rows > 0
                x[p] = r < rows ? x[p] : xn{};
            }
#pragma unroll
            for (int p = 0; p < STEPS; ++p)
                *reinterpret_cast<xn *>(tile + (p * THREADS + threadIdx.x % THREADS) * 16) = x[p];
        }
    }

    // Channels c to c + kPer - 1 of a row of d, zeros after it: what the row's last
    // chunk has of them, moved down.
    static __device__ inline auto chunk(const char *row, int c, int d)
    {
        typedef T xn __attribute__((ext_vector_type(kPer)));
        if (d < kPer) {
            xn x = {};
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (c + i < d)
                    x[i] = reinterpret_cast<const T *>(row)[c + i];
            return x;
        }
        const int at = c + kPer <= d ? c : d - kPer;
        const u32x4 raw = *reinterpret_cast<const u32x4m *>(row + at * sizeof(T));
        const unsigned __int128 x = __builtin_bit_cast(unsigned __int128, raw);
        const int down = (c - at) * int(sizeof(T)) * 8;
        return __builtin_bit_cast(xn, down < 128 ? x >> down : 0);
    }
};

// Up to 64 floats straight to LDS by a wave, zeros after n.
__device__ inline void load_floats(float *to, const float *from, int n)
{
    copy_to_lds<4>(lds_place(to), memory_rows(from, n * 4), (threadIdx.x & 63) * 4);
}

// The wave's loads to LDS have arrived (vmcnt(0)).  As a builtin, so that the
// compiler knows that its own loads have, too, and waits for none of them later,
// when the next tile's are on their way.
__device__ inline void wait_tiles()
{
    __builtin_amdgcn_s_waitcnt(0x0f70);
    asm volatile("" ::: "memory");
}

// Eight channels of the row that a lane keeps, zeros after d.
template <typename T>
__device__ inline Vec8<T> row_part(const char *row, int c, int d)
{
    typedef Tile<T, 64, 1> R;
    if constexpr (sizeof(T) == 2)
        return R::chunk(row, c, d);
    else
        return __builtin_shufflevector(R::chunk(row, c, d), R::chunk(row, c + 4, d), 0, 1, 2, 3, 4, 5, 6, 7);
}

// A operands of a tile's rows are read a good while before they are used: all of
// a product's at once, and pinned there (the compiler would read each just before
// its use and wait for it, 100 cycles and more a time).
__device__ inline void pin_reads() { __builtin_amdgcn_sched_barrier(0); }

// Operands of the scores of 32 rows from row0 on, and the scores: the products of
// a wave's columns with these rows.
template <typename T, int C, int ROWS>
struct RowOperands {
    Vec8<T> a[C / 16];

    __device__ inline void read(const char *tile, int row0)
    {
#pragma unroll
        for (int c = 0; c < C / 16; ++c)
            a[c] = Tile<T, C, ROWS>::along_channels(tile, row0, c);
    }
    __device__ inline f32x16 times(const Vec8<T> (&columns)[C / 16], f32x16 begin = f32x16{}) const
    {
        f32x16 r = product(a[0], columns[0], begin);
#pragma unroll
        for (int c = 1; c < C / 16; ++c)
            r = product(a[c], columns[c], r);
        return r;
    }
};

// Operands of the sums over 32 rows from row0 on, and the sums: sums[b] += (32
// channels of block b) x (rows), weighted by p, in two steps of 16 rows.
template <typename T, int C, int ROWS>
struct SumOperands {
    Vec8<T> a[2][C / 32];

    __device__ inline void read(const char *tile, int row0)
    {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int b = 0; b < C / 32; ++b)
                a[s][b] = Tile<T, C, ROWS>::along_rows(tile, row0 + 16 * s, b);
    }
    __device__ inline void add(f32x16 (&sums)[C / 32], int s, const f32x16 &p) const
    {
        const Vec8<T> weights = operand<T>(p, s);
#pragma unroll
        for (int b = 0; b < C / 32; ++b)
            sums[b] = product(a[s][b], weights, sums[b]);
    }
};

// Where some rows are hidden from some columns, their weight is 0, and a product
// of 0 and an infinity or NaN would be NaN.  So rows with such numbers
// (wild_rows) are added up one by one, each to the columns that see it: sees(r) for
// row r of the N from row0 on.  (A row in sight counts with a weight of 0, too,
// as it does in a tile that is seen as a whole.)  The kernels look for them before
// all else, while few registers are in use, and leave their loop for them: a branch
// inside it would cost a copy of all sums in every step.
template <typename T, int C, int ROWS, int N>
__device__ inline bool wild_rows(const char *tile, int row0)
{
    float sum = 0.f;
#pragma unroll
    for (uint32_t i = 0; i < N * Tile<T, C, ROWS>::kRow / 1024; i += sizeof(T) / 2) {
        sum = zeros_of(*reinterpret_cast<const Vec8<T> *>(tile + row0 * Tile<T, C, ROWS>::kRow + i * 1024 +
                                                          (threadIdx.x & 63) * 8 * sizeof(T)), sum);
    }
    return __ballot(sum != 0.f);
}

template <typename T, int C, int ROWS, int N, int BLOCKS, typename Sees>
__device__ inline void add_wild_rows(f32x16 (&sums)[BLOCKS], const char *tile, int row0, const f32x16 (&p)[N / 32], Sees sees)
{
    const int half = (threadIdx.x & 63) >> 5;
#pragma clang loop unroll(disable)
    for (int r = 0; r < N; ++r) {
        const int at = r / 32 * 16 + (r >> 3 & 3) * 4 + (r & 3), of = r >> 2 & 1;    // register, and half of the wave
        float w = 0.f;
#pragma unroll
        for (int j = 0; j < N / 2; ++j)
            w = at == j ? p[j / 16][j % 16] : w;
        const float across = other_half(w);
        w = of == half ? w : across;
        const bool is = sees(r);
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float x = Tile<T, C, ROWS>::at(tile, row0 + r, 32 * b + row_of(i, half));
                sums[b][i] = is ? fmaf(w, x, sums[b][i]) : sums[b][i];
                if (i % 4 == 3)         // few of these in registers at a time
                    __builtin_amdgcn_sched_barrier(0);
            }
    }
}

// ---------------------------------------------------------- who sees what --

// What a kernel needs of a call to find its rows and keys.
struct AttendShape {
    const int32_t *starts, *lengths;
    int32_t S, queries, reach, firsts;          // as in the plan
    int32_t Hl_q, Hl_kv, ratio, P, Bl, d, total;    // total: queries * ratio
    uint32_t q_token, kv_token;
    int64_t q_head, q_shard, kv_head, kv_shard;
    uint32_t pairs;                             // shards * Hl_kv
    FastDiv by_ratio, by_heads, by_Bl, by_P, by_pairs;
    float scale, scale_log2;                    // log2(e) * scale: exponents are powers of two
    float slack;                                // scores above the maximum that are not worth a rescaling
};

// The sequence of a shard, its length and the position of its first query.
struct Sequence {
    int length, start;
};

__device__ inline Sequence sequence_of(const AttendShape &A, uint32_t shard)
{
    // shards are [groups][P][Bl]
    const uint32_t rank = fastdiv(shard, A.by_Bl), b = fastdiv(rank, A.by_P) * A.Bl + (shard - rank * A.Bl);
    Sequence s;
    s.length = A.S;
    if (A.lengths) {
        const int n = scalar(A.lengths[b]);
        s.length = n < 0 ? 0 : n > A.S ? A.S : n;
    }
    s.start = A.starts ? int(scalar(A.starts[b])) : A.queries < A.S ? s.length - A.queries : 0;
    // farther out, no row has a position within the sequence either
    s.start = s.start < -A.queries ? -A.queries : s.start > A.S ? A.S : s.start;
    return s;
}

// Whether a position of the sequence sees one of its keys.
__device__ inline bool visible(const AttendShape &A, int position, int key)
{
    return key <= position && (position - key < A.reach || key < A.firsts);
}

// The keys from `first` on that a position sees, of those below `end`: offsets up
// to `last`, which come after `before` or are below `firsts`.
struct Sight {
    int last, before, firsts;

    __device__ inline Sight(const AttendShape &A, int position, int first, int end)
        : last((position < end ? position : end - 1) - first), before(position - A.reach - first), firsts(A.firsts - first)
    {
    }
    __device__ inline bool operator()(int at) const { return (at <= last) & ((at > before) | (at < firsts)); }
};

// Tiles of keys that positions [low, high] see, KEYS each: first those of the
// sinks before the window, then those of the window.
template <int KEYS>
struct KeyTiles {
    int sinks_end, window, end, sink_tiles, tiles;

    __device__ inline KeyTiles(const AttendShape &A, int low, int high)
    {
        window = low - A.reach + 1 > 0 ? low - A.reach + 1 : 0;
        end = high + 1;
        sinks_end = A.firsts < window ? A.firsts : window;
        sink_tiles = (sinks_end + KEYS - 1) / KEYS;
        tiles = high < low ? 0 : sink_tiles + (end - window + KEYS - 1) / KEYS;
    }
    __device__ inline int first(int i) const { return i < sink_tiles ? i * KEYS : window + (i - sink_tiles) * KEYS; }
    __device__ inline int rows(int i) const
    {
        const int n = (i < sink_tiles ? sinks_end : end) - first(i);
        return n < KEYS ? n : KEYS;
    }
};

// Whether all positions [low, high] of a wave see all keys [first, first + rows).
__device__ inline bool all_seen(const AttendShape &A, int low, int high, int first, int rows)
{
    const int last = first + rows - 1;
    return low <= high && last <= low && (high - first < A.reach || last < A.firsts);
}

// The positions of columns [first, first + n) that are within the sequence: their
// first and last, or last < first.
struct Span {
    int low, high;

    __device__ inline Span(const AttendShape &A, const Sequence &s, uint32_t first, uint32_t n)
    {
        const uint32_t last = first + n <= uint32_t(A.total) ? first + n - 1 : uint32_t(A.total) - 1;
        low = s.start + int(fastdiv(first, A.by_ratio));
        high = first < uint32_t(A.total) ? s.start + int(fastdiv(last, A.by_ratio)) : -1;
        low = low < 0 ? 0 : low;
        high = high < s.length ? high : s.length - 1;
    }
};

// A work-group's way through its tiles of keys and values: two of them in LDS, of
// which the next one is on its way while one is used.  What a wave does with a
// tile follows from the tile's number, and addresses go on by additions: few
// scalar instructions a tile, since a wave runs them one after another and none
// beside its vector ones.  A tile is used in parts of PART keys.
template <typename T, int C, int KEYS, int PART, int THREADS, bool DIRECT>
struct KeyWalk {
    typedef Tile<T, C, KEYS> Keys;
    char *lds;                                  // [2][2][Keys::kBytes]
    uint32_t place, token, off[Keys::kBytes / 16 / THREADS];
    int d, sinks, tiles, window, end;           // sinks: tiles of them
    int use_from, use_to, all_from, all_to;     // tiles of the window of which the wave sees some keys, and all
    bool idle;                                  // the wave sees none at all
    const char *k, *v;                          // of the next tile to fetch
    int64_t back, step;                         // from the sinks' last tile to the window's first; from tile to tile
    int fetched, fetch_left;                    // its number, and keys from it on in the sinks or the window
    int i, first, left, part;                   // of the tile in use

    __device__ inline KeyWalk(const AttendShape &A, char *lds_, const char *keys, const char *values, const Span &all,
                              const Span &mine)
        : lds(lds_), place(lds_place(lds_)), token(A.kv_token), d(A.d), k(keys), v(values)
    {
        Keys::template load_offsets<THREADS>(off, token, d);
        const KeyTiles<KEYS> t(A, all.low, all.high);
        sinks = t.sink_tiles;
        tiles = t.tiles;
        window = t.window;
        end = t.end;
        idle = mine.low > mine.high;
        // tile n of the window begins at key window + n * KEYS; where it begins
        // before the last sink, a wave sees keys before its own window
        const int behind = window < A.firsts ? 0 : mine.low - A.reach + 1 - window;
        const int ahead = mine.high - A.reach + 1 - window;
        use_from = sinks + (behind > 0 ? behind / KEYS : 0);
        use_to = sinks + (mine.high - window) / KEYS;
        all_from = sinks + (ahead > 0 ? (ahead + KEYS - 1) / KEYS : 0);
        all_to = sinks + (mine.low + 1 - window) / KEYS - 1;
        step = int64_t{KEYS} * token;
        back = (int64_t{window} - int64_t{sinks - 1} * KEYS) * token;
        first = sinks ? 0 : window;
        left = sinks ? t.sinks_end : end - window;
        k += int64_t{first} * token;
        v += int64_t{first} * token;
    }

    // The first tile on its way.
    __device__ inline void begin()
    {
        fetched = 0;
        fetch_left = left;
        i = -1;
        part = KEYS / PART;
        if (tiles)
            fetch();
    }

    __device__ inline void fetch()
    {
        const int rows = fetch_left < KEYS ? fetch_left : KEYS, buffer = (fetched & 1) * 2 * Keys::kBytes;
        Keys::template load<THREADS, DIRECT>(lds + buffer, place + buffer, off, k, token, rows, d);
        Keys::template load<THREADS, DIRECT>(lds + buffer + Keys::kBytes, place + buffer + Keys::kBytes, off, v, token, rows, d);
        ++fetched;
        const bool turn = fetched == sinks;
        k += turn ? back : step;
        v += turn ? back : step;
        fetch_left = turn ? end - window : fetch_left - KEYS;
    }

    // On to the next keys that some column of the wave sees.
    __device__ inline bool next()
    {
        if (KEYS > PART && ++part < KEYS / PART && left > part * PART)
            return true;
        part = 0;
        for (;;) {
            if (++i >= tiles)
                return false;
            if (i) {
                first = i == sinks ? window : first + KEYS;
                left = i == sinks ? end - window : left - KEYS;
            }
            wait_tiles();
            lds_barrier();          // the tile is there, and the one before is no longer read
            if (fetched < tiles)
                fetch();
            if (!idle & ((i < sinks) | ((i >= use_from) & (i <= use_to))))
                return true;
        }
    }
    __device__ inline const char *keys() const { return lds + (i & 1) * 2 * Keys::kBytes; }
    __device__ inline const char *values() const { return keys() + Keys::kBytes; }
    __device__ inline int row0() const { return KEYS > PART ? part * PART : 0; }
    __device__ inline int key() const { return first + row0(); }
    // One after the last key of the tile.
    __device__ inline int key_end() const { return first + (left < KEYS ? left : KEYS); }
    // Whether some of the tile's keys are hidden from some columns.
    __device__ inline bool hides() const { return i < sinks ? left < KEYS : (i < all_from) | (i > all_to); }
};

// A lane's column: a query and a head of the key head's group.
struct Column {
    int position;
    bool exists, live;
    uint32_t query, head;

    __device__ inline Column(const AttendShape &A, const Sequence &s, uint32_t column, uint32_t key_head)
    {
        exists = column < uint32_t(A.total);
        query = fastdiv(column, A.by_ratio);
        head = key_head * A.ratio + (column - query * A.ratio);
        position = s.start + int(query);
        live = exists && position >= 0 && position < s.length;
    }
    __device__ inline int64_t at(const AttendShape &A, uint32_t shard) const
    {
        return shard * A.q_shard + head * A.q_head + int64_t{query} * A.q_token;
    }
    __device__ inline int64_t row(const AttendShape &A, uint32_t shard) const
    {
        return (int64_t{shard} * A.Hl_q + head) * A.queries + query;
    }
};

// A row's channels as a column's operands, zeros where it is not live.
template <typename T, int C, bool DIRECT>
__device__ inline void load_column(const AttendShape &A, const char *row, bool live, Vec8<T> (&x)[C / 16])
{
    const int half = (threadIdx.x & 63) >> 5;
#pragma unroll
    for (int c = 0; c < C / 16; ++c) {
        x[c] = Vec8<T>{};
        if constexpr (DIRECT) {         // d is a multiple of a chunk, which is 8 or 4 channels
            if (sizeof(T) == 2 ? live && 16 * c + 8 * half < A.d : live && 16 * c + 8 * half + 4 < A.d)
                x[c] = *reinterpret_cast<const Vec8<T> *>(row + (16 * c + 8 * half) * sizeof(T));
            else if (sizeof(T) == 4 && live && 16 * c + 8 * half < A.d)
                x[c] = row_part<T>(row, 16 * c + 8 * half, A.d);
        } else {
            if (live)
                x[c] = row_part<T>(row, 16 * c + 8 * half, A.d);
        }
    }
}

// Work-group number `id` of `all`, so that each of the eight XCDs takes
// neighbours, which read the same keys: id % 8 is the XCD.
__device__ inline uint32_t by_xcd(uint32_t id, uint32_t all)
{
    const uint32_t x = id & 7, each = all >> 3, more = all & 7;
    return x * each + (x < more ? x : more) + (id >> 3);
}

// The pair (shard, key head) of a work-group and which of the pair's `each` it
// is, those with the most work first.  With 16-bit types an XCD takes neighbours.
// In fp32 products take so long that an XCD's reads do not matter, and all pairs'
// longest come first: 162 instead of 200 us for the gradient of three padded
// sequences of 998, 1645 instead of 1770 us for two whole ones of 2048; in bf16
// the latter take 310 us this way and 304 by XCD, 560 and 499 us with 128 channels.
struct Place {
    uint32_t pair, nth;
};

template <typename T>
__device__ inline Place place_of(const AttendShape &A, uint32_t id, uint32_t all, FastDiv by_each, uint32_t each)
{
    Place p;
    if (sizeof(T) == 4) {
        p.nth = fastdiv(id, A.by_pairs);
        p.pair = id - p.nth * A.pairs;
    } else {
        const uint32_t group = by_xcd(id, all);
        p.pair = fastdiv(group, by_each);
        p.nth = group - p.pair * each;
    }
    return p;
}

// What the wave's lanes wrote to LDS or read from it is done before what follows.
__device__ inline void wave_order()
{
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

// Weights are kept times 2^7 in fp16, of which results hold nothing: its normal
// numbers end at 2^-14 and its smallest is 2^-24, so that weights keep all bits from
// 2^-21 of the largest on and are there from 2^-31 on.  Many small weights next to a
// large one (a sink) count for as much as the large one.
template <typename T> constexpr bool kShifted = std::is_same<T, _Float16>::value;

// The exponent (to the base of 2) of a column's maximum m; where weights are shifted,
// it is rounded up.
template <typename T>
__device__ inline float top_exponent(float m, const AttendShape &A)
{
    const float top = m == -INFINITY ? 0.f : m * A.scale_log2;
    return kShifted<T> ? fmaf(fabsf(top), 0x1p-23f, top) : top;
}

// What is taken from the exponents of the column, so that the largest weight is 1, or
// where they are shifted 2^7 (2^8, where 7 is between two fp32 numbers) or less: it
// stays below 2^16 at any score.
template <typename T>
__device__ inline float weight_base(float m, const AttendShape &A)
{
    return kShifted<T> ? top_exponent<T>(m, A) - 7.f : top_exponent<T>(m, A);
}

// lse from a maximum in the scores' units and the sum relative to it (to 0 where
// no score is above -infinity).  A maximum passes over NaN, the sum does not: a row
// that sees a score of NaN has NaN.
template <typename T>
__device__ inline float log_sum(float m, float l, const AttendShape &A)
{
    return (top_exponent<T>(m, A) + __builtin_amdgcn_logf(kShifted<T> ? l * 0x1p-7f : l)) * 0.6931471805599453f;
}

// Four channels of a result's rows as stored.
template <typename T>
__device__ inline void store_four(char *row, int c, int d, const float (&x)[4])
{
    if (c + 4 <= d) {
        store_values<T, 4>(row + c * sizeof(T), x);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (c + i < d)
            reinterpret_cast<T *>(row)[c + i] = static_cast<T>(x[i]);
}

}  // namespace basp
