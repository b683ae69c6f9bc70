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

// A wave's way through tiles of ROWS keys: next() goes on to the next tile that
// some of its columns see and says whether there is one, and tile() has it.  m is
// left behind a column's maximum by up to 8 in the exponent of two, which keeps
// weights below 2^8 (in range of fp16 too) and their relative precision: after
// the first tile it hardly ever moves.  Where it does, the loop is left, the sums
// are rescaled and the tile begun again (a branch in the loop would copy them in
// every tile, see wild_rows).
template <typename T, int C, int ROWS, typename Next, typename At>
__device__ inline void attend_tiles(const AttendShape &A, const Vec8<T> (&q)[C / 16], int position, Running<C / 32> &run, Next next,
                                    At tile)
{
    const int half = (threadIdx.x & 63) >> 5;
    // half a result's scores as weights, and their sum
    const auto weigh = [&](f32x16 &s, int part, float base) {
#pragma unroll
        for (int i = 8 * part; i < 8 * part + 8; ++i) {
            s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], A.scale_log2, -base));
            run.l += s[i];
        }
    };
    bool more = next();
    while (more) {
        f32x16 s[ROWS / 32];
        float most;
        bool behind, wild;
        for (;;) {
            const auto at = tile();
#pragma unroll
            for (int t = 0; t < ROWS / 32; ++t)
                s[t] = rows_times<T, C, ROWS>(at.keys, 32 * t, q);
            if (at.part) {
                const Sight sees(A, position, at.first + at.rows);
#pragma unroll
                for (int t = 0; t < ROWS / 32; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        s[t][i] = sees(at.first + 32 * t + row_of(i, half)) ? s[t][i] : -INFINITY;
            }
            most = s[0][0];
#pragma unroll
            for (int t = 0; t < ROWS / 32; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    most = fmaxf(most, s[t][i]);
            most = fmaxf(most, other_half(most));
            behind = __ballot(most > run.m + A.slack);
            if (behind)
                break;
            wild = at.part && wild_rows<T, C, ROWS, ROWS>(at.values, 0);
            if (wild)
                break;
            // weights and their products in steps of 16 keys: exponentials are
            // taken while the matrix unit is at the step before
            const float base = run.m == -INFINITY ? 0.f : run.m * A.scale_log2;
#pragma unroll
            for (int j = 0; j < ROWS / 16; ++j) {
                weigh(s[j / 2], j % 2, base);
                const Vec8<T> weights = operand<T>(s[j / 2], j % 2);
#pragma unroll
                for (int b = 0; b < C / 32; ++b)
                    run.o[b] = product(Tile<T, C, ROWS>::along_rows(at.values, 16 * j, b), weights, run.o[b]);
            }
            more = next();
            if (!more)
                return;
        }
        if (behind) {
            run.rescale(most, A.scale_log2);
        } else {
            const float base = run.m == -INFINITY ? 0.f : run.m * A.scale_log2;
#pragma unroll
            for (int j = 0; j < ROWS / 16; ++j)
                weigh(s[j / 2], j % 2, base);
            add_wild_rows<T, C, ROWS, ROWS>(run.o, tile().values, 0, s);
            more = next();
        }
    }
}

// A tile as a wave sees it: part of the keys hidden from part of its columns, or
// not.
struct TileView {
    const char *__restrict__ keys;
    const char *__restrict__ values;
    int first, rows;
    bool part;
};

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
        D.lse[col.row(A, shard)] = col.live ? log_sum(m, total, A) : -INFINITY;
}

// 128 columns a work-group, 32 a wave; its four waves share tiles of 64 keys (32
// in fp32), of which the next one is on its way while one is used.
template <typename T, int C, bool DIRECT>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void attend_tile_kernel(const AttendDesc D)
{
    constexpr int KEYS = sizeof(T) == 2 ? 64 : 32;
    typedef Tile<T, C, KEYS> Keys;
    __shared__ __attribute__((aligned(16))) char lds[2][2][Keys::kBytes];
    const AttendShape &A = D.shape;
    const uint32_t group = by_xcd(blockIdx.x, gridDim.x), pair = fastdiv(group, D.by_blocks);
    const uint32_t block = D.blocks - 1 - (group - pair * D.blocks);       // long rows first
    const uint32_t shard = fastdiv(pair, A.by_heads), key_head = pair - shard * A.Hl_kv;
    const Sequence seq = sequence_of(A, shard);
    const uint32_t wave = scalar(threadIdx.x >> 6), lane = threadIdx.x & 63, first = block * kTileColumns;
    const Column col(A, seq, first + wave * 32 + (lane & 31), key_head);
    Vec8<T> q[C / 16];
    load_column<T, C, DIRECT>(A, D.q + col.at(A, shard), col.live, q);

    const Span all(A, seq, first, kTileColumns), mine(A, seq, first + wave * 32, 32);
    const KeyTiles<KEYS> tiles(A, all.low, all.high);

    const char *const k = D.k + shard * A.kv_shard + key_head * A.kv_head;
    const char *const v = D.v + shard * A.kv_shard + key_head * A.kv_head;
    uint32_t off[Keys::kBytes / 16 / kThreads];
    Keys::template load_offsets<kThreads>(off, A.kv_token, A.d);
    const auto fetch = [&](int i, char *to) {
        const int64_t at = int64_t{tiles.first(i)} * A.kv_token;
        Keys::template load<kThreads, DIRECT>(to, off, k + at, A.kv_token, tiles.rows(i), A.d);
        Keys::template load<kThreads, DIRECT>(to + Keys::kBytes, off, v + at, A.kv_token, tiles.rows(i), A.d);
    };
    Running<C / 32> run;
    if (tiles.tiles)
        fetch(0, lds[0][0]);
    int i = -1;
    Seen seen;
    const auto next = [&]() {
        for (++i; i < tiles.tiles; ++i) {
            wait_tiles();
            lds_barrier();          // the tile is there, and the one before is no longer read
            if (i + 1 < tiles.tiles)
                fetch(i + 1, lds[~i & 1][0]);
            seen = how_seen(A, mine.low, mine.high, tiles.first(i), tiles.rows(i));
            if (seen != Seen::none)
                return true;
        }
        return false;
    };
    attend_tiles<T, C, KEYS>(A, q, col.position, run, next, [&]() {
        return TileView{lds[i & 1][0], lds[i & 1][1], tiles.first(i), tiles.rows(i), seen == Seen::some || tiles.rows(i) < KEYS};
    });
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
        D.lse[col.row(A, shard)] = col.live ? log_sum(run.m, l, A) : -INFINITY;
}

// 32 columns a work-group; its four waves, and the work-groups of a block, take
// tiles of 32 keys in turn, each wave through LDS of its own, and join their
// sums.  For a few queries against long sequences: bound by reading the keys.
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
    const KeyTiles<KEYS> tiles(A, mine.low, mine.high);

    const char *const k = D.k + shard * A.kv_shard + key_head * A.kv_head;
    const char *const v = D.v + shard * A.kv_shard + key_head * A.kv_head;
    uint32_t off[Keys::kBytes / 16 / 64];
    Keys::template load_offsets<64>(off, A.kv_token, A.d);
    const auto fetch = [&](int i, char *to) {
        const int64_t at = int64_t{tiles.first(i)} * A.kv_token;
        Keys::template load<64, DIRECT>(to, off, k + at, A.kv_token, tiles.rows(i), A.d);
        Keys::template load<64, DIRECT>(to + Keys::kBytes, off, v + at, A.kv_token, tiles.rows(i), A.d);
    };
    Running<C / 32> run;
    const int step = D.splits * WAVES;
    int i = int(split) * WAVES + int(wave) - step, buffer = BUFFERS - 1;
    if (i + step < tiles.tiles)
        fetch(i + step, lds[wave][0][0]);
    const auto next = [&]() {
        wave_order();
        if (BUFFERS == 1 && i >= 0 && i + step < tiles.tiles)
            fetch(i + step, lds[wave][0][0]);
        i += step;
        if (i >= tiles.tiles)
            return false;
        wait_tiles();
        wave_order();
        buffer = (buffer + 1) % BUFFERS;
        if (BUFFERS == 2 && i + step < tiles.tiles)
            fetch(i + step, lds[wave][(buffer + 1) % BUFFERS][0]);
        return true;
    };
    attend_tiles<T, C, KEYS>(A, q, col.position, run, next, [&]() {
        const int first = tiles.first(i), rows = tiles.rows(i);
        return TileView{lds[wave][buffer][0], lds[wave][buffer][1], first, rows,
                        rows < KEYS || how_seen(A, mine.low, mine.high, first, rows) != Seen::all};
    });

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

// The sums of a block's work-groups, relative to the largest of their maxima.
template <typename T, int C>
__global__ __launch_bounds__(kThreads) void attend_join_kernel(const AttendDesc D)
{
    constexpr int WAVES = kThreads / 64, REGS = C / 2, SHARE = REGS / WAVES;
    const AttendShape &A = D.shape;
    const uint32_t whole = blockIdx.x, pair = fastdiv(whole, D.by_blocks), block = whole - pair * D.blocks;
    const uint32_t shard = fastdiv(pair, A.by_heads), key_head = pair - shard * A.Hl_kv;
    const Sequence seq = sequence_of(A, shard);
    const uint32_t wave = scalar(threadIdx.x >> 6), lane = threadIdx.x & 63, c = lane & 31;
    const Column col(A, seq, block * kStepColumns + c, key_head);
    const float *const from = D.partials + int64_t{whole} * D.splits * step_partial(C);
    float m = -INFINITY, total = 0.f, x[SHARE];
    for (int s = 0; s < D.splits; ++s)
        m = fmaxf(m, from[s * step_partial(C) + C * 32 + c]);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < SHARE; ++j)
        x[j] = 0.f;
    for (int s = 0; s < D.splits; ++s) {
        const float *const part = from + s * step_partial(C);
        const float factor = __builtin_amdgcn_exp2f((part[C * 32 + c] - base) * A.scale_log2);
        total += part[C * 32 + 32 + c] * factor;
#pragma unroll
        for (int j = 0; j < SHARE; ++j)
            x[j] += part[(wave * SHARE + j) * 64 + lane] * factor;
    }
    finish_columns<T, SHARE>(D, col, shard, wave * SHARE, x, m, total);
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
    return launch_kernel(reinterpret_cast<const void *>(attend_join_kernel<T, C>), dim3(uint32_t(pairs * p.blocks)), kThreads, D,
                         stream, false, true);
}

}  // namespace
}  // namespace basp

using basp::CallBuf;

extern "C" basp_status basp_attention(const basp_attention_plan *p, const void *q, const void *k, const void *v,
                                      const int32_t *starts, const int32_t *lengths, float scale, void *o, float *lse, void *ws,
                                      void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p || !(scale > 0.f) || std::isinf(scale))
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
