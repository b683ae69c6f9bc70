// attention.hip -- attention with a sliding window and sinks on head shards: the
// forward kernels and their entry point (basp.h, "Attention").
//
// One pass over the keys with the running maximum m and sum l of a softmax: a
// tile of keys gives scores s, m' = max(m, s), and o and l, kept relative to m,
// are scaled by exp(m - m') before exp(s - m') V and exp(s - m') are added.
// attention.hpp has the layouts.
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

struct AttendDesc {
    AttendShape shape;
    const char *q, *k, *v;
    char *o;
    float *lse, *partials;
    FastDiv by_blocks, by_splits;
    int32_t blocks, splits;
};

// The softmax of a wave's 32 columns as it goes: a column a lane, whose other
// rows the lane across the wave holds.  m is in the scores' units; the sum is of
// the lane's own rows.
template <int BLOCKS>
struct Running {
    float m, l;
    f32x16 o[BLOCKS];

    __device__ inline Running() : m(-INFINITY), l(0.f)
    {
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[b][i] = 0.f;
    }

    // Relative to a new maximum.
    __device__ inline void rescale(float most, float scale_log2)
    {
        const float now = fmaxf(m, most), factor = now == -INFINITY ? 1.f : __builtin_amdgcn_exp2f((m - now) * scale_log2);
        m = now;
        l *= factor;
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[b][i] *= factor;
    }
};

// The columns of a wave along its way through tiles of ROWS keys.  m is left
// behind a column's maximum by up to A.slack, about 8 in the exponent of two, which
// keeps weights in range (weight_base): after the first tile it hardly ever moves.
// Where it does, the loop is left, the sums are rescaled and the tile begun again (a
// branch in the loop would copy them in every tile, see wild_rows).
template <typename T, int C, int ROWS, typename Walk>
__device__ inline void attend_tiles(const AttendShape &A, const Vec8<T> (&q)[C / 16], int position, Running<C / 32> &run, Walk &walk)
{
    constexpr int TILES = ROWS / 32;
    const int half = (threadIdx.x & 63) >> 5;
    // half a result's scores as weights, and their sum
    const auto weigh = [&](f32x16 &s, int part, float base) {
#pragma unroll
        for (int i = 8 * part; i < 8 * part + 8; ++i) {
            s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], A.scale_log2, -base));
            run.l += s[i];
        }
    };
    wait_tiles();                   // for the columns, too, and on every way into the loop
    bool more = walk.next();
    while (more) {
        f32x16 s[TILES];
        float most;
        bool behind, wild;
        for (;;) {
            const char *const keys = walk.keys(), *const values = walk.values();
            const bool hides = walk.hides();
            wild = hides && wild_rows<T, C, ROWS, ROWS>(values, 0);
            RowOperands<T, C, ROWS> rows[TILES];
            SumOperands<T, C, ROWS> sums[TILES];
            rows[0].read(keys, 0);
            pin_reads();
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                if (t + 1 < TILES)
                    rows[t + 1].read(keys, 32 * (t + 1));
                else
                    sums[0].read(values, 0);
                s[t] = rows[t].times(q);
                pin_reads();
            }
            if (hides) {
                const Sight sees(A, position, walk.key() + 4 * half, walk.key_end());
#pragma unroll
                for (int t = 0; t < TILES; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[t][i] = sees(32 * t + row_of(i, 0)) ? s[t][i] : -INFINITY;
            }
            most = s[0][0];
#pragma unroll
            for (int t = 0; t < TILES; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    most = fmaxf(most, s[t][i]);
            most = fmaxf(most, other_half(most));
            // a sum would be rounded, by more than fp16's range allows at large scores
            behind = __ballot(kShifted<T> ? most - run.m > A.slack : most > run.m + A.slack);
            if (behind)
                break;
            if (wild)
                break;
            // weights and their products in steps of 16 keys: exponentials are
            // taken while the matrix unit is at the step before
            const float base = weight_base<T>(run.m, A);
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                if (t + 1 < TILES)
                    sums[t + 1].read(values, 32 * (t + 1));
                pin_reads();
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    weigh(s[t], j, base);
                    sums[t].add(run.o, j, s[t]);
                }
            }
            more = walk.next();
            if (!more)
                return;
        }
        if (behind) {
            run.rescale(most, A.scale_log2);
        } else {
            const float base = weight_base<T>(run.m, A);
#pragma unroll
            for (int j = 0; j < ROWS / 16; ++j)
                weigh(s[j / 2], j % 2, base);
            add_wild_rows<T, C, ROWS, ROWS>(run.o, walk.values(), 0, s, [&](int r) {
                return walk.key() + r < walk.key_end() && visible(A, position, walk.key() + r);
            });
            more = walk.next();
        }
    }
}

// SHARE registers, from number `from` on, of the finished sums of 32 columns.
template <typename T, int SHARE>
__device__ inline void finish_columns(const AttendDesc &D, const Column &col, uint32_t shard, uint32_t from, const float (&x)[SHARE],
                                      float m, float total)
{
    const AttendShape &A = D.shape;
    if (!col.exists)
        return;
    const int half = (threadIdx.x & 63) >> 5;
    const float inv = 1.f / total;
    char *const o = D.o + col.at(A, shard);
#pragma unroll
    for (int j = 0; j < SHARE; j += 4) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = col.live ? x[j + i] * inv : 0.f;
        store_four<T>(o, 32 * ((from + j) / 16) + row_of((from + j) % 16, half), A.d, y);
    }
    if (D.lse && from == 0 && half == 0)
        D.lse[col.row(A, shard)] = col.live ? log_sum<T>(m, total, A) : -INFINITY;
}

// 128 columns a work-group, 32 a wave; its four waves share tiles of 64 keys (32
// in fp32), of which the next one is on its way while one is used.  Bound by the
// issue of vector instructions, which the softmax takes more of than the matrix
// unit needs: two sequences of 16384 with a window of 1024, 32 heads of 64
// channels in bf16, take 443 us, 603 TFLOP/s; vector units busy 70% of the time,
// matrix units 36%, at the 1.8 to 1.95 GHz that the card's power leaves.  With 128
// channels matrix units are busy 48% (8192, window 2048: 630 us).  The 32 x 32
// result halves the statistics' share next to 16 x 16, and four waves to a tile
// keep reads of LDS below half of its rate.
template <typename T, int C, bool DIRECT>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 || C <= 64 ? 2 : 1) void attend_tile_kernel(const AttendDesc D)
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
    const Column col(A, seq, first + wave * 32 + (lane & 31), key_head);
    Vec8<T> q[C / 16];
    load_column<T, C, DIRECT>(A, D.q + col.at(A, shard), col.live, q);

    const Span all(A, seq, first, kTileColumns), mine(A, seq, first + wave * 32, 32);
    const int64_t at = shard * A.kv_shard + key_head * A.kv_head;
    KeyWalk<T, C, KEYS, KEYS, kThreads, DIRECT> walk(A, lds, D.k + at, D.v + at, all, mine);
    Running<C / 32> run;
    walk.begin();
    attend_tiles<T, C, KEYS>(A, q, col.position, run, walk);
    if (!col.exists)
        return;
    const float l = run.l + other_half(run.l), inv = col.live ? 1.f / l : 0.f;
    char *const o = D.o + col.at(A, shard);
    const int half = lane >> 5;
#pragma unroll
    for (int b = 0; b < C / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[j] = col.live ? run.o[b][i + j] * inv : 0.f;
            store_four<T>(o, 32 * b + row_of(i, half), A.d, x);
        }
    if (D.lse && half == 0)
        D.lse[col.row(A, shard)] = col.live ? log_sum<T>(run.m, l, A) : -INFINITY;
}

// A wave's way of its own: every step-th tile of 32 keys from number `from` on.
template <typename T, int C, int BUFFERS, bool DIRECT>
struct StepWalk {
    static constexpr int KEYS = 32;
    typedef Tile<T, C, KEYS> Keys;
    const AttendShape &A;
    const Span &mine;
    const KeyTiles<KEYS> tiles;
    char *lds;                      // [BUFFERS][2][Keys::kBytes]
    uint32_t place, off[Keys::kBytes / 16 / 64];
    const char *k, *v;
    int i, step, buffer;

    __device__ inline StepWalk(const AttendShape &shape, char *lds_, const char *keys, const char *values, const Span &span, int from,
                               int step_)
        : A(shape), mine(span), tiles(shape, span.low, span.high), lds(lds_), place(lds_place(lds_)), k(keys), v(values),
          i(from - step_), step(step_), buffer(BUFFERS - 1)
    {
        Keys::template load_offsets<64>(off, A.kv_token, A.d);
    }
    __device__ inline void fetch(int tile, int to)
    {
        const int64_t at = int64_t{tiles.first(tile)} * A.kv_token;
        const int rows = tiles.rows(tile), here = to * 2 * Keys::kBytes;
        Keys::template load<64, DIRECT>(lds + here, place + here, off, k + at, A.kv_token, rows, A.d);
        Keys::template load<64, DIRECT>(lds + here + Keys::kBytes, place + here + Keys::kBytes, off, v + at, A.kv_token, rows, A.d);
    }
    __device__ inline void begin()
    {
        if (i + step < tiles.tiles)
            fetch(i + step, 0);
    }
    __device__ inline bool next()
    {
        wave_order();
        if (BUFFERS == 1 && i >= 0 && i + step < tiles.tiles)
            fetch(i + step, 0);
        i += step;
        if (i >= tiles.tiles)
            return false;
        wait_tiles();
        wave_order();
        buffer = (buffer + 1) % BUFFERS;
        if (BUFFERS == 2 && i + step < tiles.tiles)
            fetch(i + step, (buffer + 1) % BUFFERS);
        return true;
    }
    __device__ inline const char *keys() const { return lds + buffer * 2 * Keys::kBytes; }
    __device__ inline const char *values() const { return keys() + Keys::kBytes; }
    __device__ inline int key() const { return tiles.first(i); }
    __device__ inline int key_end() const { return tiles.first(i) + tiles.rows(i); }
    __device__ inline bool hides() const
    {
        return tiles.rows(i) < KEYS || !all_seen(A, mine.low, mine.high, tiles.first(i), tiles.rows(i));
    }
};

// 32 columns a work-group; its four waves, and the work-groups of a block, take
// tiles of 32 keys in turn, each wave through LDS of its own, and join their
// sums.  For a few queries against long sequences: bound by reading the keys, so
// that waves fetch for themselves and wait for no one: 4 sequences of 65536 of a
// cache of 128 channels in fp16, 130 to 157 us, 4.9 to 6 TB/s; 16 sequences of
// 4096, 1024 in sight, 64 channels in bf16, 13 us, of which reading takes 5 and
// the rest is the chain of lengths, queries, first tile and exchange.
template <typename T, int C, bool DIRECT>
__global__ __launch_bounds__(kThreads, 1) void attend_step_kernel(const AttendDesc D)
{
    constexpr int KEYS = 32, WAVES = kThreads / 64, BUFFERS = sizeof(T) == 2 ? 2 : 1, REGS = C / 2;
    typedef Tile<T, C, KEYS> Keys;
    __shared__ __attribute__((aligned(16))) char lds[WAVES][BUFFERS][2][Keys::kBytes];
    __shared__ float all_m[WAVES][32], all_l[WAVES][32];
    const AttendShape &A = D.shape;
    const uint32_t group = by_xcd(blockIdx.x, gridDim.x), whole = fastdiv(group, D.by_splits), split = group - whole * D.splits;
    const uint32_t pair = fastdiv(whole, D.by_blocks), block = whole - pair * D.blocks;
    const uint32_t shard = fastdiv(pair, A.by_heads), key_head = pair - shard * A.Hl_kv;
    const Sequence seq = sequence_of(A, shard);
    const uint32_t wave = scalar(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const Column col(A, seq, block * kStepColumns + (lane & 31), key_head);
    Vec8<T> q[C / 16];
    load_column<T, C, DIRECT>(A, D.q + col.at(A, shard), col.live, q);
    const Span mine(A, seq, block * kStepColumns, 32);
    const int64_t at = shard * A.kv_shard + key_head * A.kv_head;
    StepWalk<T, C, BUFFERS, DIRECT> walk(A, lds[wave][0][0], D.k + at, D.v + at, mine, int(split) * WAVES + int(wave),
                                         D.splits * WAVES);
    Running<C / 32> run;
    walk.begin();
    attend_tiles<T, C, KEYS>(A, q, col.position, run, walk);

    // the waves' sums relative to the largest of their maxima
    const int half = lane >> 5, c = lane & 31;
    const float l = run.l + other_half(run.l);
    if (half == 0) {
        all_m[wave][c] = run.m;
        all_l[wave][c] = l;
    }
    lds_barrier();                  // no tile is read any more either
    float m = all_m[0][c], total = 0.f;
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
        m = fmaxf(m, all_m[w][c]);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        total += all_l[w][c] * __builtin_amdgcn_exp2f((all_m[w][c] - base) * A.scale_log2);
    const float factor = __builtin_amdgcn_exp2f((run.m - base) * A.scale_log2);
    float *const sums = reinterpret_cast<float *>(&lds[0][0][0][0]);
    static_assert(sizeof(lds) >= WAVES * REGS * 64 * 4, "the waves' sums fit");
#pragma unroll
    for (int r = 0; r < REGS; ++r)
        sums[(wave * REGS + r) * 64 + lane] = run.o[r / 16][r % 16] * factor;
    lds_barrier();
    constexpr int SHARE = REGS / WAVES;             // a wave adds up its share of the channels
    float x[SHARE];
#pragma unroll
    for (int j = 0; j < SHARE; ++j) {
        x[j] = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            x[j] += sums[(w * REGS + wave * SHARE + j) * 64 + lane];
    }
    if (D.splits > 1) {
        float *const to = D.partials + int64_t{group} * step_partial(C);
#pragma unroll
        for (int j = 0; j < SHARE; ++j)
            to[(wave * SHARE + j) * 64 + lane] = x[j];
        if (wave == 0 && half == 0) {
            to[C * 32 + c] = m;
            to[C * 32 + 32 + c] = total;
        }
        return;
    }
    finish_columns<T, SHARE>(D, col, shard, wave * SHARE, x, m, total);
}

// The sums of a block's work-groups, relative to the largest of their maxima: a
// wave takes four of a result's registers (blockIdx.y: sixteen a work-group), so
// that there are many loads at a time: 4 to 7 us, a launch and two rounds of loads.
template <typename T, int C>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(const AttendDesc D)
{
    constexpr int SHARE = 4;
    const AttendShape &A = D.shape;
    const uint32_t whole = blockIdx.x, pair = fastdiv(whole, D.by_blocks), block = whole - pair * D.blocks;
    const uint32_t shard = fastdiv(pair, A.by_heads), key_head = pair - shard * A.Hl_kv;
    const uint32_t from_reg = (blockIdx.y * (kThreads / 64) + scalar(threadIdx.x >> 6)) * SHARE;
    const uint32_t lane = threadIdx.x & 63, c = lane & 31;
    const Sequence seq = sequence_of(A, shard);
    const Column col(A, seq, block * kStepColumns + c, key_head);
    const float *const from = D.partials + int64_t{whole} * D.splits * step_partial(C);
    float m = -INFINITY, total = 0.f, x[SHARE];
#pragma unroll 8
    for (int s = 0; s < D.splits; ++s)
        m = fmaxf(m, from[s * step_partial(C) + C * 32 + c]);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < SHARE; ++j)
        x[j] = 0.f;
#pragma unroll 4
    for (int s = 0; s < D.splits; ++s) {
        const float *const part = from + s * step_partial(C);
        const float factor = __builtin_amdgcn_exp2f((part[C * 32 + c] - base) * A.scale_log2);
        total += part[C * 32 + 32 + c] * factor;
#pragma unroll
        for (int j = 0; j < SHARE; ++j)
            x[j] += part[(from_reg + j) * 64 + lane] * factor;
    }
    finish_columns<T, SHARE>(D, col, shard, from_reg, x, m, total);
}

// --------------------------------------------------------------- launches --

template <typename T, int C>
basp_status launch_attention(const basp_attention_plan &p, const AttendDesc &D, bool direct, void *stream)
{
    const int64_t pairs = int64_t{p.shards} * p.Hl_kv;
    const dim3 grid(uint32_t(pairs * p.blocks * p.splits));
    if (p.columns == kTileColumns)
        return launch_kernel(direct ? reinterpret_cast<const void *>(attend_tile_kernel<T, C, true>)
                                    : reinterpret_cast<const void *>(attend_tile_kernel<T, C, false>),
                             grid, kThreads, D, stream, true, true);
    const basp_status s = launch_kernel(direct ? reinterpret_cast<const void *>(attend_step_kernel<T, C, true>)
                                               : reinterpret_cast<const void *>(attend_step_kernel<T, C, false>),
                                        grid, kThreads, D, stream, true, p.splits == 1);
    if (s != BASP_OK || p.splits == 1)
        return s;
    return launch_kernel(reinterpret_cast<const void *>(attend_join_kernel<T, C>), dim3(uint32_t(pairs * p.blocks), C / 32), kThreads,
                         D, stream, false, true);
}

}  // namespace
}  // namespace basp

using basp::CallBuf;

extern "C" basp_status basp_attention(const basp_attention_plan *p, const void *q, const void *k, const void *v,
                                      const int32_t *starts, const int32_t *lengths, float scale, void *o, float *lse, void *ws,
                                      void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p || !basp::scale_in_range(scale))
            return BASP_ERR_INVALID;
        const int64_t nq = p->q_elems * p->es, nkv = p->kv_elems * p->es, each = int64_t{4} * p->B;
        const CallBuf in[] = {{q, nq, p->es}, {k, nkv, p->es}, {v, nkv, p->es}, {starts, starts ? each : 0, 4},
                              {lengths, lengths ? each : 0, 4}};
        const CallBuf out[] = {{o, nq, p->es}, {lse, lse ? p->lse_elems * 4 : 0, 4}, {ws, p->workspace_bytes, 16}};
        const basp_status s = basp::check_call(in, 5, out, 3);
        if (s != BASP_OK || !nq)
            return s;
        basp::AttendDesc D = {};
        D.shape = basp::attend_shape(*p, starts, lengths, scale);
        D.q = static_cast<const char *>(q);
        D.k = static_cast<const char *>(k);
        D.v = static_cast<const char *>(v);
        D.o = static_cast<char *>(o);
        D.lse = lse;
        D.partials = static_cast<float *>(ws);
        D.blocks = p->blocks;
        D.splits = p->splits;
        D.by_blocks = basp::make_fastdiv(uint32_t(p->blocks));
        D.by_splits = basp::make_fastdiv(uint32_t(p->splits));
        const bool direct = basp::whole_chunks(*p, {q, k, v});
        return BASP_BY_HEAD(basp::launch_attention, p, *p, D, direct, stream);
    });
}
