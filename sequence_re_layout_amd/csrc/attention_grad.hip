// attention_grad.hip -- the gradients of attention with a sliding window and
// sinks on head shards: kernels and entry point (basp.h, "Attention").
//
//   P = exp(s - lse),  dP = dO V^T,  dS = P (dP - delta),  delta = <dO, O>
//   dQ = scale dS K,  dK = scale dS^T Q,  dV = P^T dO
//
// Two launches that compute P and dS anew: one whose waves keep queries and
// stream keys (dQ, and delta on the way), one whose waves keep keys and stream
// the queries of their group's heads (dK, dV).  That is seven products instead
// of five, but every sum has one owner and one order: no atomics, no buffer of
// fp32 sums of dQ, and the sums over the heads of a group stay in registers.
// A block of keys with sinks is seen by all later queries; these are cut into
// chunks of a work-group each, whose sums a third launch adds in their order;
// other blocks, too, where there are few work-groups.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attention.hpp"
#include "attention_launch.hpp"
#include "index_plan.hpp"
#include "plan_internal.hpp"
#include "runtime.hpp"

namespace basp {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
// Whether scores begin from -lse / scale in the gradients of k and v (QueryWalk).
template <typename T> constexpr bool kFromLse = sizeof(T) == 2;

constexpr int kFewTiles = 3;        // tiles of keys up to which <dO, O> is summed again from P and dP

// P, at most 1 here, is taken times 2^12 in the products of the gradient of V in
// fp16: it keeps all bits from 2^-26 on, where 50000 equal weights are below fp16's
// normal numbers as they are.  2^4 is left for the rounding of large scores.
template <typename T> constexpr float kWeightExponent = kShifted<T> ? 12.f : 0.f;
template <typename T> constexpr float kOneWeight = kShifted<T> ? 0x1p-12f : 1.f;

// dS may have any size next to dout: P is small where a row sees many keys.  In
// fp16 it is rounded times a power of two, which the sums are freed of at the end.
// In the gradient of q that is a column's own.  The sizes of its dO and of the first
// values give one, no less than 1, that hardly ever has to move: all bits are kept
// where P is 2^-22 and more.  It comes down where a |dS| is above 2^15, so that
// nothing overflows.  A wave leaves the largest |dS| and |dO| of its 32 columns for
// the gradients of k and v, which take the power of a chunk's queries from them, so
// that their largest dS is 2^14 to 2^15: all bits are kept down to 2^-28 of it.  dS
// are computed anew there, and where dP is about delta (a row of one key) they are
// what is left of its rounding, at most 4 (d + 2) 2^-24 times d products of dO and V:
// the power keeps these in range, too.  (To find it on the way there takes more
// registers than there are: 1350 us instead of 1120 for two sequences of 8192, 128
// channels and a window of 2048.)
//
// The power that takes numbers of exponent `of` to `to`, 2^60 at most.
__device__ inline float power_for(int to, int of) { return __builtin_amdgcn_ldexpf(1.f, to - of < 60 ? to - of : 60); }

// The largest of `most` and a lane's numbers.
__device__ inline float largest(const f32x16 &x, float most)
{
#pragma unroll
    for (int i = 0; i < 16; ++i)
        most = fmaxf(most, fabsf(x[i]));
    return most;
}

template <typename T, int N>
__device__ inline float largest(const Vec8<T> (&x)[N])
{
    float most = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            most = fmaxf(most, fabsf(static_cast<float>(x[n][i])));
    return most;
}

// Whether it is to come down; infinities stay, such sums have no finite value.
__device__ inline bool too_large(float most) { return most > 0x1p15f && most < INFINITY; }

// The exponent of two of a positive number.
__device__ inline int exponent_of(float x) { return int(__builtin_bit_cast(uint32_t, x) >> 23) - 127; }

template <int BLOCKS>
__device__ inline void times(f32x16 (&sums)[BLOCKS], float factor)
{
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sums[b][i] *= factor;
}

// The largest of a wave's finite numbers that are not below 0.
__device__ inline float largest_of_wave(float x)
{
    x = x < INFINITY ? x : 0.f;
#pragma unroll
    for (int far = 1; far < 64; far *= 2)
        x = fmaxf(x, __shfl_xor(x, far));
    return x;
}

struct AttendGradDesc {
    AttendShape shape;
    const char *q, *k, *v, *o, *dout;
    const float *lse;
    char *dq, *dk, *dv;
    float *rows, *partials;         // rows: [2][lse_elems], -lse / scale (or log2(e) * -lse) and -delta
    float *most;                    // in fp16: [pairs][units][2], the largest |dS| and |dO| of 32 columns
    int64_t lse_elems;
    FastDiv by_blocks, by_items, by_sink_chunks, by_chunks, by_sink_cuts, by_cuts;
    int32_t heads;                  // of a group, that a work-group of the gradient of keys and values takes
    // chunks: of a block, in all; cuts: of its queries
    int32_t blocks, units, items, sink_blocks, sink_chunk, sink_chunks, sink_cuts, chunk, chunks, cuts, key_blocks;
};

// 128 columns (queries and heads) a work-group, 32 a wave; tiles of keys and
// values as in the forward pass.  Three products a tile: matrix units are busy
// half of the time, next to the exponents and the reads of both forms of the keys
// from LDS (two sequences of 8192 with a window of 2048, 32 heads of 128 channels
// in bf16: 790 us).
template <typename T, int C, bool DIRECT>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 || C <= 64 ? 2 : 1) void attend_dq_kernel(const AttendGradDesc D)
{
    constexpr int KEYS = sizeof(T) == 2 ? 64 : 32;
    typedef Tile<T, C, KEYS> Keys;
    __shared__ __attribute__((aligned(16))) char lds[4 * Keys::kBytes];
    const AttendShape &A = D.shape;
    const Place place = place_of<T>(A, blockIdx.x, gridDim.x, D.by_blocks, D.blocks);
    const uint32_t pair = place.pair, block = D.blocks - 1 - place.nth;    // later queries see more
    const uint32_t shard = fastdiv(pair, A.by_heads), key_head = pair - shard * A.Hl_kv;
    const Sequence seq = sequence_of(A, shard);
    const uint32_t wave = scalar(threadIdx.x >> 6), lane = threadIdx.x & 63, first = block * kTileColumns;
    const int half = lane >> 5;
    const Column col(A, seq, first + wave * 32 + (lane & 31), key_head);
    Vec8<T> q[C / 16], g[C / 16];
    load_column<T, C, DIRECT>(A, D.q + col.at(A, shard), col.live, q);
    load_column<T, C, DIRECT>(A, D.dout + col.at(A, shard), col.live, g);
    const float lse_at = col.live ? D.lse[col.row(A, shard)] : 0.f, lse = lse_at * kLog2e;

    const Span all(A, seq, first, kTileColumns), mine(A, seq, first + wave * 32, 32);
    const int64_t at = shard * A.kv_shard + key_head * A.kv_head;
    KeyWalk<T, C, KEYS, 32, kThreads, DIRECT> walk(A, lds, D.k + at, D.v + at, all, mine);
    // P and dP of the next 32 keys; P is 0 where a key is hidden
    const auto weigh = [&](const auto &at, f32x16 &p, f32x16 &dp) {
        RowOperands<T, C, KEYS> keys, values;
        keys.read(at.keys(), at.row0());
        pin_reads();
        values.read(at.values(), at.row0());
        p = keys.times(q);
        pin_reads();
        dp = values.times(g);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            p[i] = __builtin_amdgcn_exp2f(fmaf(p[i], A.scale_log2, -lse));
        if (at.hides()) {
            const Sight sees(A, col.position, at.key() + 4 * half, at.key_end());
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool is = sees(row_of(i, 0));
                p[i] = is ? p[i] : 0.f;
                dp[i] = is ? dp[i] : 0.f;
            }
        }
    };

    // delta = <dO, O> = sum P dP.  O has been rounded to its type, which shows
    // where a row sees few keys: there delta is summed first, in fp32.
    float delta = 0.f;
    if (walk.tiles <= kFewTiles) {
        auto once = walk;
        once.begin();
        wait_tiles();
        while (once.next()) {
            f32x16 p, dp;
            weigh(once, p, dp);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                delta = fmaf(p[i], dp[i], delta);
        }
        lds_barrier();
    } else if (col.live) {
        const char *const o = D.o + col.at(A, shard);
#pragma unroll
        for (int c = 0; c < C / 16; ++c) {
            const Vec8<T> x = row_part<T>(o, 16 * c + 8 * half, A.d);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                delta = fmaf(static_cast<float>(x[i]), static_cast<float>(g[c][i]), delta);
        }
    }
    delta += other_half(delta);
    if (col.live && half == 0) {
        D.rows[col.row(A, shard)] = kFromLse<T> ? -lse_at / A.scale : -lse;
        D.rows[D.lse_elems + col.row(A, shard)] = -delta;
    }

    f32x16 sums[C / 32];
#pragma unroll
    for (int b = 0; b < C / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sums[b][i] = 0.f;
    walk.begin();
    wait_tiles();                   // for the columns, too, and on every way into the loop
    bool more = walk.next();
    float power = 1.f, most = 0.f;
    const int64_t unit = int64_t{pair} * D.units + first / 32 + wave;
    const bool leaves = lane == 0 && first / 32 + wave < uint32_t(D.units);
    if constexpr (kShifted<T>) {
        const Vec8<T> some[1] = {*reinterpret_cast<const Vec8<T> *>(walk.values() + lane * 16)};
        float of_g = largest<T>(g), of_v = largest<T>(some);
        of_g = fmaxf(of_g, other_half(of_g));
        const float of_all = largest_of_wave(of_g);
        if (leaves)
            D.most[unit * 2 + 1] = of_all;
        power = fmaxf(1.f, power_for(8, exponent_of(of_g) + exponent_of(more ? largest_of_wave(of_v) : 0.f)));
        delta *= power;
    }
    while (more) {
        f32x16 ds[1];
        bool beyond = false;
        for (;;) {
            f32x16 dp;
            const bool wild = walk.hides() && wild_rows<T, C, KEYS, 32>(walk.keys(), walk.row0());
            weigh(walk, ds[0], dp);
            SumOperands<T, C, KEYS> operands;
            operands.read(walk.keys(), walk.row0());
            pin_reads();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                ds[0][i] *= kShifted<T> ? fmaf(dp[i], power, -delta) : dp[i] - delta;
            if constexpr (kShifted<T>) {
                most = largest(ds[0], most);
                beyond = __ballot(too_large(most));
            }
            if (beyond | wild)
                break;
            operands.add(sums, 0, ds[0]);
            operands.add(sums, 1, ds[0]);
            more = walk.next();
            if (!more)
                break;
        }
        if (beyond) {               // a lane and its opposite alike, and then these keys again
            most = fmaxf(most, other_half(most));
            const float down = too_large(most) ? __builtin_amdgcn_ldexpf(1.f, 7 - exponent_of(most)) : 1.f;
            power *= down;
            delta *= down;
            most *= down;
            times(sums, down);
        } else if (more) {
            add_wild_rows<T, C, KEYS, 32>(sums, walk.keys(), walk.row0(), ds, [&](int r) {
                return walk.key() + r < walk.key_end() && visible(A, col.position, walk.key() + r);
            });
            more = walk.next();
        }
    }
    if constexpr (kShifted<T>) {
        const float here = largest_of_wave(most / power);
        if (leaves)
            D.most[unit * 2] = here;
        times(sums, 1.f / power);
    }
    if (!col.exists)
        return;
    char *const dq = D.dq + col.at(A, shard);
#pragma unroll
    for (int b = 0; b < C / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = col.live ? sums[b][i + j] * A.scale : 0.f;
            store_four<T>(dq, 32 * b + row_of(i, half), A.d, x);
        }
}

// N registers of a result's column of keys as stored, the first ones of `channel` on.
template <typename T, int N, typename Sums>
__device__ inline void store_key(const AttendShape &A, char *to, uint32_t shard, uint32_t key_head, int key, int channel, int half,
                                 const Sums &sums, float scale)
{
    if (key >= A.S)
        return;
    char *const row = to + shard * A.kv_shard + key_head * A.kv_head + int64_t{key} * A.kv_token;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = sums[i + j] * scale;
        store_four<T>(row, channel + row_of(i, half), A.d, x);
    }
}

// A work-group's way through the queries [begin, end) of each head of a group and
// their gradients, as KeyWalk's through keys: tiles of ROWS in LDS, used in parts
// of 32, with two numbers of each query.  The products begin from -lse / scale and
// -delta instead of 0, so that P = exp(scale * result) and dS = P * result.  In fp32
// the first would round every step of a product at lse's size instead of the score's
// (3000 equal keys of 128 channels: dv off by 2.5e-6 of it, 7e-7 this way): there
// log2(e) * -lse is added afterwards.
template <typename T, int C, int ROWS, bool DIRECT>
struct QueryWalk {
    typedef Tile<T, C, ROWS> Rows;
    char *lds;                                  // [2][2][Rows::kBytes]
    float *lds_rows;                            // [2][2][64]
    uint32_t place, token, off[Rows::kBytes / 16 / kThreads];
    int d, count, tiles, all;                   // queries, and tiles of a head and of all heads
    int use_from, use_to, all_from, all_to;     // parts of a head in which some query sees some of the wave's keys, and all all
    int start;                                  // position of the first query
    const char *q, *g;                          // of the next tile to fetch
    const float *numbers;                       // of its first query: for the scores (first wave), or -delta (second)
    int64_t step, turn;                         // from tile to tile, and from a head's last to the next one's first
    int queries, fetched, fetch_left;
    int i, in_head, left, part;

    __device__ inline QueryWalk(const AttendShape &A, char *lds_, float *lds_rows_, const AttendGradDesc &D, int64_t at, int64_t row,
                                int first_position, int begin, int end, int heads, int key)
        : lds(lds_), lds_rows(lds_rows_), place(lds_place(lds_)), token(A.q_token), d(A.d)
    {
        Rows::template load_offsets<kThreads>(off, token, d);
        count = end - begin;
        tiles = count > 0 ? (count + ROWS - 1) / ROWS : 0;
        all = tiles * heads;
        start = first_position + begin;
        queries = A.queries;
        // part n of a head holds positions start + 32 * n to start + 32 * n + 31, the
        // wave keys `key` to key + 31
        use_from = (key - 31 - start + 31) >> 5;
        use_to = key < A.firsts ? 0x7fffffff : (A.reach - 1 + key + 31 - start) >> 5;
        all_from = (key + 31 - start + 31) >> 5;
        all_to = key + 31 < A.firsts ? 0x7fffffff : (A.reach - 1 + key - 31 - start) >> 5;
        step = int64_t{ROWS} * token;
        turn = A.q_head - int64_t{tiles - 1} * step;
        q = D.q + at + int64_t{begin} * token;
        g = D.dout + at + int64_t{begin} * token;
        numbers = D.rows + scalar(threadIdx.x >> 6) * D.lse_elems + row + begin;
    }
    __device__ inline void begin()
    {
        fetched = 0;
        fetch_left = count;
        i = -1;
        in_head = -1;
        left = 0;
        part = ROWS / 32;
        if (all)
            fetch();
    }
    __device__ inline void fetch()
    {
        const int rows = fetch_left < ROWS ? fetch_left : ROWS, buffer = fetched & 1, at = buffer * 2 * Rows::kBytes;
        Rows::template load<kThreads, DIRECT>(lds + at, place + at, off, q, token, rows, d);
        Rows::template load<kThreads, DIRECT>(lds + at + Rows::kBytes, place + at + Rows::kBytes, off, g, token, rows, d);
        const uint32_t wave = scalar(threadIdx.x >> 6);
        if (wave < 2)
            load_floats(lds_rows + (buffer * 2 + wave) * 64, numbers, rows);
        ++fetched;
        const bool last = fetch_left <= ROWS;
        q += last ? turn : step;
        g += last ? turn : step;
        numbers += last ? queries - (tiles - 1) * ROWS : ROWS;
        fetch_left = last ? count : fetch_left - ROWS;
    }
    // On to the next 32 queries of which some see some key of the wave.
    __device__ inline bool next()
    {
        for (;;) {
            if (ROWS > 32 && ++part < ROWS / 32 && left > part * 32) {
                ++in_head;
            } else {
                part = 0;
                if (++i >= all)
                    return false;
                left -= ROWS;
                ++in_head;
                if (left <= 0) {
                    left = count;
                    in_head = 0;
                }
                wait_tiles();
                lds_barrier();
                if (fetched < all)
                    fetch();
            }
            if ((in_head >= use_from) & (in_head <= use_to))
                return true;
        }
    }
    __device__ inline const char *queries_at() const { return lds + (i & 1) * 2 * Rows::kBytes; }
    __device__ inline const char *grads() const { return queries_at() + Rows::kBytes; }
    __device__ inline int row0() const { return ROWS > 32 ? part * 32 : 0; }
    __device__ inline int position() const { return start + 32 * in_head; }
    __device__ inline int rows() const { return left - row0(); }
    // The numbers of the rows of a result's registers, and of four of them from j on.
    typedef float x4 __attribute__((ext_vector_type(4)));
    __device__ inline x4 four_numbers(int which, int half, int j) const
    {
        return *reinterpret_cast<const x4 *>(lds_rows + (i & 1) * 128 + which * 64 + row0() + 4 * half + row_of(j, 0));
    }
    __device__ inline f32x16 numbers_at(int which, int half) const
    {
        f32x16 r;
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const x4 x = four_numbers(which, half, j);
            r[j] = x[0];
            r[j + 1] = x[1];
            r[j + 2] = x[2];
            r[j + 3] = x[3];
        }
        return r;
    }
    __device__ inline f32x16 lse(int half) const { return numbers_at(0, half); }
    __device__ inline f32x16 delta(int half) const { return numbers_at(1, half); }
    __device__ inline bool hides() const { return (in_head < all_from) | (in_head > all_to) | (rows() < 32); }
};

// 128 keys a work-group, 32 a wave, and a chunk of the queries that see them,
// head by head of the group: tiles of 64 queries (32 in fp32) and their gradients
// go through LDS, the next one on its way while one is used.  Where the keys'
// sums take half of the registers that two waves of a SIMD have (16-bit types,
// over 64 channels), the values are kept in LDS instead, and tiles are of 32
// queries to leave room for them.  Four products a tile, and what it reads from
// LDS is as much for each wave: two sequences of 8192 with a window of 2048, 32
// heads of 128 channels in bf16, 1100 us with matrix units busy 48% of the time,
// 1467 us with the values in registers, some of which were spilled.
template <typename T, int C, bool DIRECT>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 || C <= 64 ? 2 : 1) void attend_dkv_kernel(const AttendGradDesc D)
{
    constexpr bool VALUES_IN_LDS = sizeof(T) == 2 && C > 64;
    constexpr int ROWS = sizeof(T) == 2 && !VALUES_IN_LDS ? 64 : 32;
    typedef Tile<T, C, ROWS> Rows;
    typedef Tile<T, C, kKeyBlock> Values;
    __shared__ __attribute__((aligned(16))) char lds_values[VALUES_IN_LDS ? Values::kBytes : 16];
    __shared__ __attribute__((aligned(16))) char lds[4 * Rows::kBytes];
    __shared__ __attribute__((aligned(16))) float lds_rows[2 * 2 * 64];
    const AttendShape &A = D.shape;
    const Place place = place_of<T>(A, blockIdx.x, gridDim.x, D.by_items, D.items);
    const uint32_t pair = place.pair, item = place.nth;
    const uint32_t shard = fastdiv(pair, A.by_heads), key_head = pair - shard * A.Hl_kv;
    const uint32_t in_sinks = uint32_t(D.sink_blocks) * D.sink_chunks;
    const bool sinks = item < in_sinks;
    const uint32_t nth = sinks ? item : item - in_sinks, of = fastdiv(nth, sinks ? D.by_sink_chunks : D.by_chunks);
    const int part = int(nth - of * (sinks ? D.sink_chunks : D.chunks)), key_block = int(of) + (sinks ? 0 : D.sink_blocks);
    const Sequence seq = sequence_of(A, shard);
    const uint32_t wave = scalar(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5, wave_key = key_block * kKeyBlock + int(wave) * 32, key = wave_key + int(lane & 31);
    const bool exists = key < seq.length;

    Vec8<T> k[C / 16], v[VALUES_IN_LDS ? 1 : C / 16];
    const int64_t at_key = shard * A.kv_shard + key_head * A.kv_head + int64_t{exists ? key : 0} * A.kv_token;
    load_column<T, C, DIRECT>(A, D.k + at_key, exists, k);
    if constexpr (VALUES_IN_LDS) {
        const int first = key_block * kKeyBlock, rows = seq.length - first < kKeyBlock ? seq.length - first : kKeyBlock;
        uint32_t off[Values::kBytes / 16 / kThreads];
        Values::template load_offsets<kThreads>(off, A.kv_token, A.d);
        if (rows > 0)
            Values::template load<kThreads, DIRECT>(lds_values, lds_place(lds_values), off,
                                                    D.v + shard * A.kv_shard + key_head * A.kv_head + int64_t{first} * A.kv_token,
                                                    A.kv_token, rows, A.d);
    } else {
        load_column<T, C, DIRECT>(A, D.v + at_key, exists, v);
    }
    f32x16 dk[C / 32], dv[C / 32];
#pragma unroll
    for (int b = 0; b < C / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            dk[b][i] = dv[b][i] = 0.f;

    // the chunk's queries
    const int last_key = key_block * kKeyBlock + kKeyBlock - 1;
    int begin = key_block * kKeyBlock - seq.start, end = seq.length - seq.start;
    begin = begin < 0 ? 0 : begin;
    end = end < A.queries ? end : A.queries;
    if (!sinks)
        end = end < last_key + A.reach - seq.start ? end : last_key + A.reach - seq.start;
    const int length = sinks ? D.sink_chunk : D.chunk;
    const int head_part = fastdiv(part, sinks ? D.by_sink_cuts : D.by_cuts);
    begin += (part - head_part * (sinks ? D.sink_cuts : D.cuts)) * length;
    end = end < begin + length ? end : begin + length;
    const int head = key_head * A.ratio + head_part * D.heads;
    QueryWalk<T, C, ROWS, DIRECT> walk(A, lds, lds_rows, D, shard * A.q_shard + head * A.q_head,
                                       (int64_t{shard} * A.Hl_q + head) * A.queries, seq.start, begin, end, D.heads, wave_key);
    walk.begin();
    float power = 1.f;
    if constexpr (kShifted<T>) {
        float of_v;
        if constexpr (VALUES_IN_LDS) {
            Vec8<T> mine[C / 16];
            load_column<T, C, DIRECT>(A, D.v + at_key, exists, mine);
            of_v = largest<T>(mine);
        } else {
            of_v = largest<T>(v);
        }
        const uint32_t units_end = end > begin ? (uint32_t(end) * A.ratio + 31) / 32 : 0;
        float most = 0.f, of_g = 0.f;
        for (uint32_t u = uint32_t(begin) * A.ratio / 32 + lane; u < units_end; u += 64) {
            const float *const from = D.most + (int64_t{pair} * D.units + u) * 2;
            most = fmaxf(most, from[0]);
            of_g = fmaxf(of_g, from[1]);
        }
        const int largest_ds = exponent_of(largest_of_wave(most));
        const int rounding = exponent_of(largest_of_wave(of_g)) + exponent_of(largest_of_wave(of_v)) - 7;
        power = power_for(14, int(scalar(uint32_t(largest_ds > rounding ? largest_ds : rounding))));
    }
    const float factor = kOneWeight<T> * power;     // from weights as they are taken to those of dS
    wait_tiles();                   // for the keys, too, and on every way into the loop
    bool more = walk.next();
    while (more) {
        f32x16 p[1], ds[1];
        for (;;) {
            const char *const queries = walk.queries_at(), *const grads = walk.grads();
            const int row0 = walk.row0();
            const bool wild = walk.hides() && (wild_rows<T, C, ROWS, 32>(queries, row0) || wild_rows<T, C, ROWS, 32>(grads, row0));
            // Operands are read a stage of products ahead; 32 registers of them
            // where the values are in LDS, so that nothing is spilled: a register
            // that comes back from memory would wait for the tile on its way.
            constexpr int HALF = VALUES_IN_LDS ? C / 32 : 1;
            Vec8<T> one[HALF], other[HALF];
            RowOperands<T, C, ROWS> of_queries, of_grads;
            SumOperands<T, C, ROWS> operands;
            if constexpr (VALUES_IN_LDS) {
                const int mine = int(wave) * 32;
                const uint32_t here = lane_here();
                f32x16 s = walk.lse(half), dp;
#pragma unroll
                for (int c = 0; c < HALF; ++c)
                    one[c] = Rows::along_channels(queries, row0, c, here);
                pin_reads();
#pragma unroll
                for (int c = 0; c < HALF; ++c) {
                    s = product(one[c], k[c], s);
                    one[c] = Rows::along_channels(queries, row0, HALF + c, here);
                }
                pin_reads();
#pragma unroll
                for (int c = 0; c < HALF; ++c) {
                    s = product(one[c], k[HALF + c], s);
                    if (c == 0)
                        dp = walk.delta(half);
                    one[c] = Rows::along_channels(grads, row0, c, here);
                    other[c] = Values::along_channels(lds_values, mine, c, here);
                }
                pin_reads();
#pragma unroll
                for (int c = 0; c < HALF; ++c) {
                    dp = product(one[c], other[c], dp);
                    one[c] = Rows::along_channels(grads, row0, HALF + c, here);
                    other[c] = Values::along_channels(lds_values, mine, HALF + c, here);
                }
                pin_reads();
#pragma unroll
                for (int c = 0; c < HALF; ++c) {
                    dp = product(one[c], other[c], dp);
                    one[c] = Rows::along_rows(grads, row0, c, here);
                    other[c] = Rows::along_rows(grads, row0 + 16, c, here);
                }
                pin_reads();
                p[0] = s;
                ds[0] = dp;
            } else {
                of_queries.read(queries, row0);
                pin_reads();
                of_grads.read(grads, row0);
                p[0] = of_queries.times(k, kFromLse<T> ? walk.lse(half) : f32x16{});
                pin_reads();
                ds[0] = of_grads.times(v, walk.delta(half));
                if constexpr (kFromLse<T>)
                    operands.read(grads, row0);
                pin_reads();
            }
            if constexpr (kFromLse<T>) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    p[0][i] = __builtin_amdgcn_exp2f(kShifted<T> ? fmaf(p[0][i], A.scale_log2, kWeightExponent<T>) : p[0][i] * A.scale_log2);
                    ds[0][i] *= kShifted<T> ? p[0][i] * factor : p[0][i];
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const auto lse = walk.four_numbers(0, half, j);
#pragma unroll
                    for (int i = j; i < j + 4; ++i) {
                        p[0][i] = __builtin_amdgcn_exp2f(fmaf(p[0][i], A.scale_log2, lse[i - j]));
                        ds[0][i] *= p[0][i];
                    }
                    pin_reads();        // few of these in registers at a time
                }
            }
            if (walk.hides()) {
                // the rows from `first` on that see the key: up to `last`
                const int first = walk.position() + 4 * half, from = key - first, rows = walk.rows() - 4 * half;
                const int last = key < A.firsts ? rows - 1 : key + A.reach - 1 - first < rows - 1 ? key + A.reach - 1 - first : rows - 1;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const bool is = (row_of(i, 0) >= from) & (row_of(i, 0) <= last);
                    p[0][i] = is ? p[0][i] : 0.f;
                    ds[0][i] = is ? ds[0][i] : 0.f;
                }
            }
            if (wild)
                break;
            if constexpr (VALUES_IN_LDS) {
                const uint32_t here = lane_here();
                const Vec8<T> p0 = operand<T>(p[0], 0), p1 = operand<T>(p[0], 1);
#pragma unroll
                for (int c = 0; c < HALF; ++c) {
                    dv[c] = product(one[c], p0, dv[c]);
                    one[c] = Rows::along_rows(queries, row0, c, here);
                }
#pragma unroll
                for (int c = 0; c < HALF; ++c) {
                    dv[c] = product(other[c], p1, dv[c]);
                    other[c] = Rows::along_rows(queries, row0 + 16, c, here);
                }
                pin_reads();
                const Vec8<T> ds0 = operand<T>(ds[0], 0), ds1 = operand<T>(ds[0], 1);
#pragma unroll
                for (int c = 0; c < HALF; ++c)
                    dk[c] = product(one[c], ds0, dk[c]);
#pragma unroll
                for (int c = 0; c < HALF; ++c)
                    dk[c] = product(other[c], ds1, dk[c]);
            } else {
                if constexpr (!kFromLse<T>)     // registers are few, and the products long
                    operands.read(grads, row0);
                operands.add(dv, 0, p[0]);
                operands.add(dv, 1, p[0]);
                operands.read(queries, row0);
                operands.add(dk, 0, ds[0]);
                operands.add(dk, 1, ds[0]);
            }
            more = walk.next();
            if (!more)
                break;
        }
        if (more) {
            const auto sees = [&](int r) { return r < walk.rows() && visible(A, walk.position() + r, key); };
            add_wild_rows<T, C, ROWS, 32>(dv, walk.grads(), walk.row0(), p, sees);
            add_wild_rows<T, C, ROWS, 32>(dk, walk.queries_at(), walk.row0(), ds, sees);
            more = walk.next();
        }
    }
    if constexpr (kShifted<T>)
        times(dk, 1.f / power);
    if ((sinks ? D.sink_chunks : D.chunks) == 1) {
#pragma unroll
        for (int b = 0; b < C / 32; ++b) {
            store_key<T, 16>(A, D.dk, shard, key_head, key, 32 * b, half, dk[b], A.scale);
            store_key<T, 16>(A, D.dv, shard, key_head, key, 32 * b, half, dv[b], kOneWeight<T>);
        }
        return;
    }
    // unfinished blocks of a pair: those with sinks, if they are cut, then the others
    const int64_t before = D.sink_chunks > 1 ? in_sinks : 0;
    const int64_t each = before + (D.chunks > 1 ? int64_t{D.key_blocks - D.sink_blocks} * D.chunks : 0);
    float *const to = D.partials + (pair * each + (sinks ? 0 : before) + nth) * (2 * kKeyBlock * C);
#pragma unroll
    for (int b = 0; b < C / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            to[((0 + wave) * (C / 2) + b * 16 + i) * 64 + lane] = dk[b][i];
            to[((4 + wave) * (C / 2) + b * 16 + i) * 64 + lane] = dv[b][i];
        }
}

struct AttendJoinDesc {
    AttendShape shape;
    const float *partials;
    char *dk, *dv;
    int64_t pair_stride;            // numbers from one pair's to the next one's
    FastDiv by_blocks;
    int32_t blocks, first_block;    // unfinished blocks of a pair, of which the first
    int32_t sink_blocks, sink_chunks, chunks;       // blocks of sink_chunks chunks, then of `chunks`
};

// The sums of a block of keys over its chunks: a wave takes 32 keys and 16
// channels of dK or dV, four chunks on their way at a time.  13 us for the 44 MB of
// chunks of three fp32 sequences of 998, whose 96 blocks have 6 or 16 of them.
template <typename T, int C>
__global__ __launch_bounds__(kThreads) void attend_grad_join_kernel(const AttendJoinDesc D)
{
    const AttendShape &A = D.shape;
    constexpr int EACH = 2 * kKeyBlock * C, AHEAD = 4;
    const uint32_t pair = fastdiv(blockIdx.x, D.by_blocks), block = blockIdx.x - pair * D.blocks;
    const uint32_t shard = fastdiv(pair, A.by_heads), key_head = pair - shard * A.Hl_kv;
    const uint32_t unit = blockIdx.y * (kThreads / 64) + scalar(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t part = unit % (C / 16), wave = unit / (C / 16);         // wave: 0 to 3 of dK, 4 to 7 of dV
    const bool sinks = block < uint32_t(D.sink_blocks);
    const int64_t before = sinks ? int64_t{block} * D.sink_chunks
                                 : int64_t{D.sink_blocks} * D.sink_chunks + int64_t{block - D.sink_blocks} * D.chunks;
    const int chunks = sinks ? D.sink_chunks : D.chunks;
    const float *from = D.partials + pair * D.pair_stride + before * EACH + (wave * (C / 2) + part * 8) * 64 + lane;
    float sums[8] = {};
    for (int c = 0; c < chunks; c += AHEAD, from += AHEAD * EACH) {
        float x[AHEAD][8];
#pragma unroll
        for (int n = 0; n < AHEAD; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[n][i] = c + n < chunks ? from[n * EACH + i * 64] : 0.f;
#pragma unroll
        for (int n = 0; n < AHEAD; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                sums[i] += x[n][i];
    }
    const int key = int(D.first_block + block) * kKeyBlock + int(wave & 3) * 32 + int(lane & 31);
    store_key<T, 8>(A, wave < 4 ? D.dk : D.dv, shard, key_head, key, int(part) * 16, int(lane >> 5), sums,
                    wave < 4 ? A.scale : kOneWeight<T>);
}

// --------------------------------------------------------------- launches --

template <typename T, int C>
basp_status launch_attention_grad(const basp_attention_plan &p, const AttendGradDesc &D, bool direct, void *stream)
{
    const int64_t pairs = int64_t{p.shards} * p.Hl_kv;
    const bool cut[2] = {p.sink_blocks && p.sink_chunks > 1, p.chunks > 1 && p.key_blocks > p.sink_blocks};
    basp_status s = launch_kernel(direct ? reinterpret_cast<const void *>(attend_dq_kernel<T, C, true>)
                                         : reinterpret_cast<const void *>(attend_dq_kernel<T, C, false>),
                                  dim3(uint32_t(pairs * D.blocks)), kThreads, D, stream, true, false);
    if (s == BASP_OK)
        s = launch_kernel(direct ? reinterpret_cast<const void *>(attend_dkv_kernel<T, C, true>)
                                 : reinterpret_cast<const void *>(attend_dkv_kernel<T, C, false>),
                          dim3(uint32_t(pairs * D.items)), kThreads, D, stream, false, !cut[0] && !cut[1]);
    if (s == BASP_OK && (cut[0] || cut[1])) {
        AttendJoinDesc J = {};
        J.shape = D.shape;
        J.partials = D.partials;
        J.dk = D.dk;
        J.dv = D.dv;
        J.sink_blocks = cut[0] ? p.sink_blocks : 0;
        J.blocks = J.sink_blocks + (cut[1] ? p.key_blocks - p.sink_blocks : 0);
        J.by_blocks = make_fastdiv(uint32_t(J.blocks));
        J.first_block = cut[0] ? 0 : p.sink_blocks;
        J.sink_chunks = p.sink_chunks;
        J.chunks = p.chunks;
        J.pair_stride = (int64_t{J.sink_blocks} * J.sink_chunks + int64_t{J.blocks - J.sink_blocks} * J.chunks) * (2 * kKeyBlock * C);
        s = launch_kernel(reinterpret_cast<const void *>(attend_grad_join_kernel<T, C>),
                          dim3(uint32_t(pairs * J.blocks), 4 * (C / 32)), kThreads, J, stream, false, true);
    }
    return s;
}

}  // namespace
}  // namespace basp

using basp::CallBuf;

extern "C" basp_status basp_attention_grad(const basp_attention_plan *p, const void *q, const void *k, const void *v, const void *o,
                                           const float *lse, const void *dout, const int32_t *starts, const int32_t *lengths,
                                           float scale, void *dq, void *dk, void *dv, void *ws, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p || !basp::scale_in_range(scale))
            return BASP_ERR_INVALID;
        const int64_t nq = p->q_elems * p->es, nkv = p->kv_elems * p->es, each = int64_t{4} * p->B;
        const CallBuf in[] = {{q, nq, p->es}, {k, nkv, p->es}, {v, nkv, p->es}, {o, nq, p->es}, {lse, p->lse_elems * 4, 4},
                              {dout, nq, p->es}, {starts, starts ? each : 0, 4}, {lengths, lengths ? each : 0, 4}};
        const CallBuf out[] = {{dq, nq, p->es}, {dk, nkv, p->es}, {dv, nkv, p->es}, {ws, p->grad_workspace_bytes, 16}};
        const basp_status s = basp::check_call(in, 8, out, 4);
        if (s != BASP_OK || !nq)
            return s;
        basp::AttendGradDesc D = {};
        D.shape = basp::attend_shape(*p, starts, lengths, scale);
        D.q = static_cast<const char *>(q);
        D.k = static_cast<const char *>(k);
        D.v = static_cast<const char *>(v);
        D.o = static_cast<const char *>(o);
        D.dout = static_cast<const char *>(dout);
        D.lse = lse;
        D.dq = static_cast<char *>(dq);
        D.dk = static_cast<char *>(dk);
        D.dv = static_cast<char *>(dv);
        D.rows = static_cast<float *>(ws);
        D.partials = reinterpret_cast<float *>(static_cast<char *>(ws) + p->partials_at);
        D.most = D.rows + 2 * p->lse_elems;
        D.units = p->grad_units;
        D.lse_elems = p->lse_elems;
        D.blocks = p->grad_blocks;
        D.by_blocks = basp::make_fastdiv(uint32_t(p->grad_blocks));
        D.sink_blocks = p->sink_blocks;
        D.sink_chunk = p->sink_chunk;
        D.sink_chunks = p->sink_chunks;
        D.chunk = p->chunk;
        D.chunks = p->chunks;
        D.sink_cuts = p->sink_chunks / p->head_parts;
        D.cuts = p->chunks / p->head_parts;
        D.heads = p->ratio / p->head_parts;
        D.by_sink_cuts = basp::make_fastdiv(uint32_t(D.sink_cuts));
        D.by_cuts = basp::make_fastdiv(uint32_t(D.cuts));
        D.key_blocks = p->key_blocks;
        D.items = p->sink_blocks * p->sink_chunks + (p->key_blocks - p->sink_blocks) * p->chunks;
        D.by_items = basp::make_fastdiv(uint32_t(D.items));
        D.by_sink_chunks = basp::make_fastdiv(uint32_t(p->sink_chunks));
        D.by_chunks = basp::make_fastdiv(uint32_t(p->chunks));
        const bool direct = basp::whole_chunks(*p, {q, k, v, dout});
        return BASP_BY_HEAD(basp::launch_attention_grad, p, *p, D, direct, stream);
    });
}
