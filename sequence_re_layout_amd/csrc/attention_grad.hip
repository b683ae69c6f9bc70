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
// chunks of a work-group each, whose sums a third launch adds in their order.
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
constexpr int kFewTiles = 3;        // tiles of keys up to which <dO, O> is summed again from P and dP

struct AttendGradDesc {
    AttendShape shape;
    const char *q, *k, *v, *o, *dout;
    const float *lse;
    char *dq, *dk, *dv;
    float *rows, *partials;         // rows: [2][lse_elems], lse in powers of two, and delta
    int64_t lse_elems;
    FastDiv by_blocks, by_items, by_sink_chunks, by_chunks;
    int32_t blocks, items, sink_blocks, sink_chunk, sink_chunks, chunk, chunks, key_blocks;
};

// 128 columns (queries and heads) a work-group, 32 a wave; tiles of keys and
// values as in the forward pass.
template <typename T, int C, bool DIRECT>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) void attend_dq_kernel(const AttendGradDesc D)
{
    constexpr int KEYS = sizeof(T) == 2 ? 64 : 32, PARTS = KEYS / 32;
    typedef Tile<T, C, KEYS> Keys;
    __shared__ __attribute__((aligned(16))) char lds[2][2][Keys::kBytes];
    const AttendShape &A = D.shape;
    const uint32_t group = by_xcd(blockIdx.x, gridDim.x), pair = fastdiv(group, D.by_blocks);
    const uint32_t block = D.blocks - 1 - (group - pair * D.blocks);       // long rows first
    const uint32_t shard = fastdiv(pair, A.by_heads), key_head = pair - shard * A.Hl_kv;
    const Sequence seq = sequence_of(A, shard);
    const uint32_t wave = scalar(threadIdx.x >> 6), lane = threadIdx.x & 63, first = block * kTileColumns;
    const int half = lane >> 5;
    const Column col(A, seq, first + wave * 32 + (lane & 31), key_head);
    Vec8<T> q[C / 16], g[C / 16];
    load_column<T, C, DIRECT>(A, D.q + col.at(A, shard), col.live, q);
    load_column<T, C, DIRECT>(A, D.dout + col.at(A, shard), col.live, g);
    const float lse = col.live ? D.lse[col.row(A, shard)] * kLog2e : 0.f;

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
    // on to the next 32 keys that some column of the wave sees
    int u = -1;
    Seen seen;
    const auto next = [&]() {
        for (++u; u < tiles.tiles * PARTS; ++u) {
            const int j = u / PARTS, t = u % PARTS, rows = tiles.rows(j) - 32 * t;
            if (t == 0) {
                wait_tiles();
                lds_barrier();
                if (j + 1 < tiles.tiles)
                    fetch(j + 1, lds[~j & 1][0]);
            }
            seen = rows > 0 ? how_seen(A, mine.low, mine.high, tiles.first(j) + 32 * t, rows < 32 ? rows : 32) : Seen::none;
            if (seen != Seen::none)
                return true;
        }
        return false;
    };
    // P and dP of these keys; P is 0 where a key is hidden
    const auto weigh = [&](f32x16 &p, f32x16 &dp) {
        const int j = u / PARTS, t = u % PARTS, from = tiles.first(j) + 32 * t, rows = tiles.rows(j) - 32 * t;
        p = rows_times<T, C, KEYS>(lds[j & 1][0], 32 * t, q);
        dp = rows_times<T, C, KEYS>(lds[j & 1][1], 32 * t, g);
#pragma unroll
        for (int i = 0; i < 16; ++i)
            p[i] = __builtin_amdgcn_exp2f(fmaf(p[i], A.scale_log2, -lse));
        const bool part = seen == Seen::some || rows < 32;
        if (part) {
            const Sight sees(A, col.position, from + rows);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool is = sees(from + row_of(i, half));
                p[i] = is ? p[i] : 0.f;
                dp[i] = is ? dp[i] : 0.f;
            }
        }
        return part;
    };

    // delta = <dO, O> = sum P dP.  O has been rounded to its type, which shows
    // where a row sees few keys: there delta is summed first, in fp32.
    float delta = 0.f;
    if (tiles.tiles <= kFewTiles) {
        if (tiles.tiles)
            fetch(0, lds[0][0]);
        while (next()) {
            f32x16 p, dp;
            weigh(p, dp);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                delta = fmaf(p[i], dp[i], delta);
        }
        u = -1;
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
        D.rows[col.row(A, shard)] = lse;
        D.rows[D.lse_elems + col.row(A, shard)] = delta;
    }

    f32x16 sums[C / 32];
#pragma unroll
    for (int b = 0; b < C / 32; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sums[b][i] = 0.f;
    if (tiles.tiles)
        fetch(0, lds[0][0]);
    bool more = next();
    while (more) {
        f32x16 ds[1];
        for (;;) {
            f32x16 dp;
            const bool part = weigh(ds[0], dp);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                ds[0][i] *= dp[i] - delta;
            const char *const keys = lds[u / PARTS & 1][0];
            if (part && wild_rows<T, C, KEYS, 32>(keys, u % PARTS * 32))
                break;
            add_rows<T, C, KEYS, 32>(sums, keys, u % PARTS * 32, ds);
            more = next();
            if (!more)
                break;
        }
        if (more) {
            add_wild_rows<T, C, KEYS, 32>(sums, lds[u / PARTS & 1][0], u % PARTS * 32, ds);
            more = next();
        }
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

// Sixteen channels of a result's column of keys as stored.
template <typename T>
__device__ inline void store_key(const AttendShape &A, char *to, uint32_t shard, uint32_t key_head, int key, int block, int half,
                                 const f32x16 &sums, float scale)
{
    if (key >= A.S)
        return;
    char *const row = to + shard * A.kv_shard + key_head * A.kv_head + int64_t{key} * A.kv_token;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = sums[i + j] * scale;
        store_four<T>(row, 32 * block + row_of(i, half), A.d, x);
    }
}

// 128 keys a work-group, 32 a wave, and a chunk of the queries that see them,
// head by head of the group: tiles of 64 queries (32 in fp32) and their
// gradients go through LDS, the next one on its way while one is used.
template <typename T, int C, bool DIRECT>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 && C <= 64 ? 2 : 1) void attend_dkv_kernel(const AttendGradDesc D)
{
    constexpr int ROWS = sizeof(T) == 2 ? 64 : 32, PARTS = ROWS / 32;
    typedef Tile<T, C, ROWS> Rows;
    __shared__ __attribute__((aligned(16))) char lds[2][2][Rows::kBytes];
    __shared__ __attribute__((aligned(16))) float lds_rows[2][2][64];
    const AttendShape &A = D.shape;
    const uint32_t group = by_xcd(blockIdx.x, gridDim.x), pair = fastdiv(group, D.by_items), item = group - pair * D.items;
    const uint32_t shard = fastdiv(pair, A.by_heads), key_head = pair - shard * A.Hl_kv;
    const uint32_t in_sinks = uint32_t(D.sink_blocks) * D.sink_chunks;
    const bool sinks = item < in_sinks;
    const uint32_t nth = sinks ? item : item - in_sinks, of = fastdiv(nth, sinks ? D.by_sink_chunks : D.by_chunks);
    const int part = int(nth - of * (sinks ? D.sink_chunks : D.chunks)), key_block = int(of) + (sinks ? 0 : D.sink_blocks);
    const Sequence seq = sequence_of(A, shard);
    const uint32_t wave = scalar(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int half = lane >> 5, wave_key = key_block * kKeyBlock + int(wave) * 32, key = wave_key + int(lane & 31);
    const bool exists = key < seq.length;

    Vec8<T> k[C / 16], v[C / 16];
    const int64_t at_key = shard * A.kv_shard + key_head * A.kv_head + int64_t{exists ? key : 0} * A.kv_token;
    load_column<T, C, DIRECT>(A, D.k + at_key, exists, k);
    load_column<T, C, DIRECT>(A, D.v + at_key, exists, v);
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
    begin += part * length;
    end = end < begin + length ? end : begin + length;
    const int tiles = end > begin ? (end - begin + ROWS - 1) / ROWS : 0, all = tiles * A.ratio;

    uint32_t off[Rows::kBytes / 16 / kThreads];
    Rows::template load_offsets<kThreads>(off, A.q_token, A.d);
    const auto fetch = [&](int head, int tile, int buffer) {
        char *const to = lds[buffer][0];
        const int from = begin + tile * ROWS, rows = end - from < ROWS ? end - from : ROWS;
        const uint32_t q_head = key_head * A.ratio + head;
        const int64_t at = shard * A.q_shard + q_head * A.q_head + int64_t{from} * A.q_token;
        Rows::template load<kThreads, DIRECT>(to, off, D.q + at, A.q_token, rows, A.d);
        Rows::template load<kThreads, DIRECT>(to + Rows::kBytes, off, D.dout + at, A.q_token, rows, A.d);
        if (wave < 2)
            load_floats(lds_rows[buffer][wave], D.rows + wave * D.lse_elems + (int64_t{shard} * A.Hl_q + q_head) * A.queries + from,
                        rows);
    };
    if (all)
        fetch(0, 0, 0);
    // on to the next 32 queries that see some key of the wave
    int u = -1, at = 0, tile = 0, head = 0;
    Seen seen;
    const auto next = [&]() {
        for (++u; u < all * PARTS; ++u) {
            const int j = u / PARTS, t = u % PARTS;
            if (t == 0) {
                wait_tiles();
                lds_barrier();
                at = begin + tile * ROWS;
                tile = tile + 1 < tiles ? tile + 1 : 0;
                head += tile == 0;
                if (j + 1 < all)
                    fetch(head, tile, ~j & 1);
            } else {
                at += 32;
            }
            const int low = seq.start + at, high = seq.start + (at + 32 < end ? at + 32 : end) - 1;
            seen = how_seen(A, low, high, wave_key, 32);
            if (seen != Seen::none)
                return true;
        }
        return false;
    };
    bool more = next();
    while (more) {
        f32x16 p[1], ds[1];
        for (;;) {
            const int buffer = u / PARTS & 1, row0 = u % PARTS * 32, rows = end - at;
            const char *const queries = lds[buffer][0], *const grads = lds[buffer][1];
            p[0] = rows_times<T, C, ROWS>(queries, row0, k);
            ds[0] = rows_times<T, C, ROWS>(grads, row0, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = row0 + row_of(i, half);
                p[0][i] = __builtin_amdgcn_exp2f(fmaf(p[0][i], A.scale_log2, -lds_rows[buffer][0][row]));
                ds[0][i] = p[0][i] * (ds[0][i] - lds_rows[buffer][1][row]);
            }
            const bool part = seen == Seen::some || rows < 32;
            if (part) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int row = row_of(i, half);
                    const bool is = (row < rows) & Sight(A, seq.start + at + row, A.S)(key);
                    p[0][i] = is ? p[0][i] : 0.f;
                    ds[0][i] = is ? ds[0][i] : 0.f;
                }
                if (wild_rows<T, C, ROWS, 32>(queries, row0) || wild_rows<T, C, ROWS, 32>(grads, row0))
                    break;
            }
            add_rows<T, C, ROWS, 32>(dv, grads, row0, p);
            add_rows<T, C, ROWS, 32>(dk, queries, row0, ds);
            more = next();
            if (!more)
                break;
        }
        if (more) {
            add_wild_rows<T, C, ROWS, 32>(dv, lds[u / PARTS & 1][1], u % PARTS * 32, p);
            add_wild_rows<T, C, ROWS, 32>(dk, lds[u / PARTS & 1][0], u % PARTS * 32, ds);
            more = next();
        }
    }
    if ((sinks ? D.sink_chunks : D.chunks) == 1) {
#pragma unroll
        for (int b = 0; b < C / 32; ++b) {
            store_key<T>(A, D.dk, shard, key_head, key, b, half, dk[b], A.scale);
            store_key<T>(A, D.dv, shard, key_head, key, b, half, dv[b], 1.f);
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
    const float *partials;          // of the first pair's first block of these
    char *dk, *dv;
    int64_t pair_stride;            // numbers from one pair's to the next one's
    FastDiv by_blocks;
    int32_t blocks, first_block, chunks;
};

// The sums of a block of keys over its chunks: a wave takes 32 keys and 32
// channels of dK or dV.
template <typename T, int C>
__global__ __launch_bounds__(kThreads) void attend_grad_join_kernel(const AttendJoinDesc D)
{
    const AttendShape &A = D.shape;
    const uint32_t pair = fastdiv(blockIdx.x, D.by_blocks), block = blockIdx.x - pair * D.blocks;
    const uint32_t shard = fastdiv(pair, A.by_heads), key_head = pair - shard * A.Hl_kv;
    const uint32_t unit = blockIdx.y * (kThreads / 64) + scalar(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const uint32_t b = unit % (C / 32), wave = unit / (C / 32);            // wave: 0 to 3 of dK, 4 to 7 of dV
    const float *from = D.partials + pair * D.pair_stride + int64_t{block} * D.chunks * (2 * kKeyBlock * C) +
                        (wave * (C / 2) + b * 16) * 64 + lane;
    f32x16 sums;
#pragma unroll
    for (int i = 0; i < 16; ++i)
        sums[i] = 0.f;
    for (int c = 0; c < D.chunks; ++c, from += 2 * kKeyBlock * C)
#pragma unroll
        for (int i = 0; i < 16; ++i)
            sums[i] += from[i * 64];
    const int key = int(D.first_block + block) * kKeyBlock + int(wave & 3) * 32 + int(lane & 31);
    store_key<T>(A, wave < 4 ? D.dk : D.dv, shard, key_head, key, int(b), int(lane >> 5), sums, wave < 4 ? A.scale : 1.f);
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
    const int64_t numbers = 2 * kKeyBlock * C, sink_part = p.sink_chunks > 1 ? int64_t{p.sink_blocks} * p.sink_chunks : 0;
    const int64_t part = p.chunks > 1 ? int64_t{p.key_blocks - p.sink_blocks} * p.chunks : 0;
    for (int i = 0; i < 2 && s == BASP_OK; ++i) {
        if (!cut[i])
            continue;
        AttendJoinDesc J = {};
        J.shape = D.shape;
        J.partials = D.partials + (i ? sink_part : 0) * numbers;
        J.dk = D.dk;
        J.dv = D.dv;
        J.pair_stride = (sink_part + part) * numbers;
        J.blocks = i ? p.key_blocks - p.sink_blocks : p.sink_blocks;
        J.by_blocks = make_fastdiv(uint32_t(J.blocks));
        J.first_block = i ? p.sink_blocks : 0;
        J.chunks = i ? p.chunks : p.sink_chunks;
        s = launch_kernel(reinterpret_cast<const void *>(attend_grad_join_kernel<T, C>),
                          dim3(uint32_t(pairs * J.blocks), 2 * (C / 32)), kThreads, J, stream, false, i == 1 || !cut[1]);
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
        if (!p || !(scale > 0.f) || std::isinf(scale))
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
        D.lse_elems = p->lse_elems;
        D.blocks = p->grad_blocks;
        D.by_blocks = basp::make_fastdiv(uint32_t(p->grad_blocks));
        D.sink_blocks = p->sink_blocks;
        D.sink_chunk = p->sink_chunk;
        D.sink_chunks = p->sink_chunks;
        D.chunk = p->chunk;
        D.chunks = p->chunks;
        D.key_blocks = p->key_blocks;
        D.items = p->sink_blocks * p->sink_chunks + (p->key_blocks - p->sink_blocks) * p->chunks;
        D.by_items = basp::make_fastdiv(uint32_t(D.items));
        D.by_sink_chunks = basp::make_fastdiv(uint32_t(p->sink_chunks));
        D.by_chunks = basp::make_fastdiv(uint32_t(p->chunks));
        const bool direct = basp::whole_chunks(*p, {q, k, v, dout});
        return BASP_BY_HEAD(basp::launch_attention_grad, p, *p, D, direct, stream);
    });
}
