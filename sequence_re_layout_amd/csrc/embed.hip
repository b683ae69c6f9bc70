// embed.hip -- embedding lookup into the sequence-sharded layout and its
// gradient by sorted tokens: kernels and entry points of the embedding plans
// (basp.h, "Index-driven re-layouts").
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#define BASP_HD __host__ __device__
#include "index_plan.hpp"
#include "plan_internal.hpp"
#include "rowvec.hpp"
#include "runtime.hpp"
#include "sort.hpp"

namespace basp {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kLaunchVectors = int64_t{1} << 30;

// Token t's id, or V where it names no row of the table (or the one left out).
__device__ inline uint32_t row_of_id(const void *ids, int64_t t, int64_t V, int64_t without, int wide)
{
    const int64_t id = wide ? static_cast<const int64_t *>(ids)[t] : static_cast<const int32_t *>(ids)[t];
    return uint32_t(id >= 0 && id < V && id != without ? id : V);
}

struct LookupDesc {
    const void *ids;                // of the whole call, as out
    const char *table;
    char *out;
    int64_t t0, nvec;               // first token and vectors of this launch
    int64_t V;
    uint32_t row;
    FastDiv per_row;
    basp_seq_order order;
    float scale;
    int32_t wide_ids;
};

// Each lane reads one vector of a table row, scales it in fp32 and writes it
// to the token's place.  UNI: a row is a whole number of waves.  Bound by HBM:
// 32768 tokens x 2048, 183 MB in 31 us (5.9 TB/s); the table is read with plain
// loads, since frequent ids come again.
template <typename E, int VW, bool UNI>
__global__ __launch_bounds__(kThreads) void lookup_kernel(const LookupDesc D)
{
    constexpr int N = VW / sizeof(E);
    const uint32_t v = blockIdx.x * kThreads + threadIdx.x;
    if (v >= D.nvec)
        return;
    uint32_t t = fastdiv(v, D.per_row);
    if constexpr (UNI)
        t = scalar(t);
    const uint32_t off = vec_offset<VW>(v - t * D.per_row.d, D.row);
    const uint32_t token = uint32_t(D.t0) + t;
    const uint32_t id = row_of_id(D.ids, token, D.V, -1, D.wide_ids);
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = 0.f;
    if (id < D.V) {
        unpack<E, VW>(load_vec<VW, false>(D.table + uint64_t(id) * D.row + off), f);
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] *= D.scale;
    }
    store_vec<VW>(D.out + uint64_t(seq_row(D.order, token)) * D.row + off, pack<E, VW>(f));
}

// ----------------------------------------------- rows that no token names --

// While a token's id is first read, its number is left at tags[id].  A row of
// the table has a token if and only if its tag is a token with that id,
// whatever the tags held before and whichever token wrote last: no memory has
// to be cleared for this, and no sorted list searched.
struct ZeroDesc {
    const void *ids;
    uint32_t *tags;
    char *dtable;
    int64_t T, V, padding;
    int32_t wide_ids;
    ZeroPieces z;                   // rows of this launch
};

template <int WAVES>
__device__ inline void zero_unnamed(const ZeroDesc &D, uint32_t group)
{
    write_zeros<WAVES>(D.dtable, D.z, group, [&](uint32_t r) {
        const uint32_t t = D.T ? D.tags[r] : 0;
        return t >= D.T || row_of_id(D.ids, t, D.V, D.padding, D.wide_ids) != r;
    });
}

// ------------------------------------------------------- tokens by their id --

// One pass of the sort by id, least significant digit first.  The launches
// of a pass are bound by latency and use a few work-groups; the others write
// rows of zeros meanwhile, which is what the whole call spends most on where
// the table is larger than the batch.
struct PassDesc {
    const uint32_t *keys_in, *tokens_in;
    uint32_t *keys_out, *tokens_out;
    int32_t *hist;
    int64_t items;
    int32_t first, shift, bins;
    int32_t groups;                 // work-groups of the pass
    ZeroDesc zero;
};

__device__ inline uint32_t pass_key(const PassDesc &D, int64_t i)
{
    return D.first ? row_of_id(D.zero.ids, i, D.zero.V, D.zero.padding, D.zero.wide_ids) : D.keys_in[i];
}

__global__ __launch_bounds__(kSortBlock) void digit_count_kernel(const PassDesc D)
{
    extern __shared__ int lds[];
    if (blockIdx.x >= uint32_t(D.groups)) {
        zero_unnamed<kSortWaves>(D.zero, blockIdx.x - D.groups);
        return;
    }
    const int64_t T = D.zero.T, begin = blockIdx.x * D.items, end = begin + D.items < T ? begin + D.items : T;
    sort_count<kSortWaves>(lds, begin, end, D.bins, D.hist + int64_t{blockIdx.x} * D.bins, [&](int64_t i) {
        const uint32_t key = pass_key(D, i);
        if (D.first && key < D.zero.V)
            D.zero.tags[key] = uint32_t(i);
        return int(key >> D.shift) & (D.bins - 1);
    });
}

template <int R>
__global__ __launch_bounds__(kSortBlock) void digit_place_kernel(const PassDesc D)
{
    extern __shared__ int lds[];
    if (blockIdx.x >= uint32_t(D.groups)) {
        zero_unnamed<kSortWaves>(D.zero, blockIdx.x - D.groups);
        return;
    }
    const int64_t T = D.zero.T, begin = blockIdx.x * D.items, end = begin + D.items < T ? begin + D.items : T;
    sort_place<kSortWaves, R>(
        sort_lds(lds, kSortWaves, D.bins), begin, end, D.bins, 1, D.hist, D.groups, blockIdx.x,
        [&](int64_t i) -> uint64_t {
            return uint64_t(D.first ? uint32_t(i) : D.tokens_in[i]) << 32 | pass_key(D, i);
        },
        [&](uint64_t pair) { return int(uint32_t(pair) >> D.shift) & (D.bins - 1); },
        [&](int64_t, uint64_t pair, int at) {
            if (at >= 0 && at < T) {
                D.keys_out[at] = uint32_t(pair);
                D.tokens_out[at] = uint32_t(pair >> 32);
            }
        });
}

// A small sort in one launch, by counting: a token's place is the number of
// (id, token) pairs below its own.  Every work-group holds all T pairs in LDS
// and places kRankTokens of them: a lane compares one of its tokens with every
// kRankParts-th vector of pairs.  T^2 comparisons cost less than the launches
// of the general sort up to kRankNarrow tokens.  Pair: the pairs as whole
// numbers id * T + token, which 32 bits hold for most plans.
constexpr int kRankThreads = 1024, kRankTokens = 16, kRankParts = kRankThreads / kRankTokens;

struct RankDesc {
    uint32_t *keys, *tokens;
    ZeroDesc zero;                  // ids and tags
};

template <typename Pair>
size_t rank_lds_bytes(int64_t T)
{
    constexpr int64_t STEP = kRankParts * (16 / sizeof(Pair));
    return size_t((T + STEP - 1) / STEP * STEP) * sizeof(Pair);
}

template <typename Pair>
__global__ __launch_bounds__(kRankThreads) void rank_kernel(const RankDesc D)
{
    constexpr int N = 16 / sizeof(Pair), STEP = kRankParts * N;
    typedef Pair vec __attribute__((ext_vector_type(N)));
    extern __shared__ uint4 rank_lds[];
    __shared__ int place[kRankTokens];
    const vec *const pairs = reinterpret_cast<const vec *>(rank_lds);
    Pair *const one = reinterpret_cast<Pair *>(rank_lds);
    const int T = int(D.zero.T), first = blockIdx.x * kRankTokens;
    const int filled = (T + STEP - 1) / STEP * STEP;
    for (int i = threadIdx.x; i < filled; i += kRankThreads) {
        Pair p = ~Pair{0};
        if (i < T) {
            const uint32_t key = row_of_id(D.zero.ids, i, D.zero.V, D.zero.padding, D.zero.wide_ids);
            p = Pair(key) * Pair(T) + Pair(i);
            if (i >= first && i < first + kRankTokens && key < D.zero.V)
                D.zero.tags[key] = uint32_t(i);
        }
        one[i] = p;
    }
    if (threadIdx.x < kRankTokens)
        place[threadIdx.x] = 0;
    lds_barrier();
    const int token = threadIdx.x % kRankTokens;
    const Pair mine = one[first + token < T ? first + token : first];
    int below = 0;
#pragma unroll 4
    for (int i = threadIdx.x / kRankTokens; i < filled / N; i += kRankParts) {
        const vec p = pairs[i];
#pragma unroll
        for (int n = 0; n < N; ++n)
            below += p[n] < mine;
    }
    below += __shfl_xor(below, 16);
    below += __shfl_xor(below, 32);
    if ((threadIdx.x & 63) < kRankTokens)
        atomicAdd(&place[token], below);
    lds_barrier();
    if (threadIdx.x < kRankTokens && first + token < T) {
        D.keys[place[token]] = uint32_t(mine / Pair(T));
        D.tokens[place[token]] = uint32_t(first + token);
    }
}

// ------------------------------------------------------- sums by their id --

struct GradDesc {
    const uint32_t *keys, *tokens;  // sorted
    const char *dout;
    char *dtable;
    float *partials;                // [blocks][2][width]
    int64_t T, width, block_tokens;
    uint32_t V, blocks, row, vecs, grad_row, elems;
    FastDiv col_groups;
    int32_t lanes_log2, chunk;
    uint32_t sum_groups;            // work-groups that sum; the others write zeros
    basp_seq_order order;
    float scale;
    ZeroDesc zero;
};

// The channels of vector a of table row `key`, scaled: written, or with ACC
// added to what is there.
template <typename G, bool ACC, int N>
__device__ inline void write_grad(const GradDesc &D, uint32_t key, uint32_t a, const float (&sum)[N])
{
    const uint32_t first = a * N, last = D.elems - N, at = first < last ? first : last;
    char *p = D.dtable + uint64_t(key) * D.grad_row + uint64_t(at) * sizeof(G);
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = sum[i] * D.scale;
    if constexpr (ACC) {
        if (at != first) {             // the vector before adds the channels both hold
            for (int i = int(first - at); i < N; ++i) {
                G *q = reinterpret_cast<G *>(p) + i;
                *q = static_cast<G>(static_cast<float>(*q) + f[i]);
            }
            return;
        }
        float old[N];
        load_values<G, N>(p, old);
#pragma unroll
        for (int i = 0; i < N; ++i)
            f[i] += old[i];
    }
    store_values<G, N>(p, f);
}

template <int N>
__device__ inline void clear(float (&f)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = 0.f;
}

template <int N>
__device__ inline void add(float (&f)[N], const float (&g)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] += g[i];
}

constexpr uint32_t kNoKey = 0xffffffffu;    // no id: V is at most 2^30

// The sorted tokens, `chunk` to a team of lanes; up to kMerge teams of a work-
// group that follow each other make a block.  A lane adds one vector of
// channels over its team's chunk and writes the sum wherever the id changes.
// The sum of an id that reaches over an end of the chunk goes to LDS, where
// the block's first team joins them; one that reaches over an end of the
// block's tokens leaves an fp32 partial sum in each block: slot 0 where it
// began in an earlier one, slot 1 where it begins in this one.
// UNI: teams are whole waves; the chunk's ids and rows are loaded at once, one
// token a lane, and read from there as scalars.
// Why chunks: an id's tokens may be one or all, and either way a team adds
// `chunk` rows, 8 loads in flight (16 spill into memory: 164 against 130 us for
// the whole call).  32768 tokens x 2048 into 131072 rows: 216 MB in 41 us
// without the zeros (5.3 TB/s).
template <typename E, typename G, int VW, bool UNI, bool ACC>
__global__ __launch_bounds__(kSumThreads) void chunk_sum_kernel(const GradDesc D)
{
    constexpr int N = VW / sizeof(E), U = 8;
    constexpr int HEAD = 1, ON = 2, TAIL = 4;  // of a team: a sum that began before its chunk, one that
                                               // goes on from there behind it, one that begins in it and goes on
    __shared__ float sums[2][kSumThreads][N];
    __shared__ uint32_t key_of[2][UNI ? 4 : kSumThreads];
    __shared__ int state[UNI ? 4 : kSumThreads];
    if (blockIdx.x >= D.sum_groups) {
        zero_unnamed<kSumThreads / 64>(D.zero, blockIdx.x - D.sum_groups);
        return;
    }
    const int lanes_log2 = UNI ? 6 : D.lanes_log2, lanes = 1 << lanes_log2, teams = kSumThreads >> lanes_log2;
    const int lane = threadIdx.x & (lanes - 1);
    int team = threadIdx.x >> lanes_log2;
    if constexpr (UNI)
        team = scalar(team);
    const uint32_t group = fastdiv(blockIdx.x, D.col_groups);
    const uint32_t a = (blockIdx.x - group * D.col_groups.d) * lanes + lane;
    const bool live = a < D.vecs;
    const uint32_t off = vec_offset<VW>(live ? a : 0, D.row);
    const int64_t begin = (int64_t{group} * teams + team) * D.chunk;
    const int n = begin >= D.T ? 0 : D.T - begin < D.chunk ? int(D.T - begin) : D.chunk;

    uint32_t my_key = D.V, my_row = 0;          // UNI: of the chunk's token number `lane`
    if constexpr (UNI)
        if (lane < n) {
            my_key = D.keys[begin + lane];
            my_row = seq_row(D.order, D.tokens[begin + lane]);
        }
    const uint32_t before = n && begin ? D.keys[begin - 1] : kNoKey;
    const uint32_t after = n && begin + n < D.T ? D.keys[begin + n] : kNoKey;
    const auto key_at = [&](int j) -> uint32_t {
        if constexpr (UNI)
            return __builtin_amdgcn_readlane(my_key, j);
        return D.keys[begin + j];
    };
    const auto row_at = [&](int j) -> uint32_t {
        if constexpr (UNI)
            return __builtin_amdgcn_readlane(my_row, j);
        return seq_row(D.order, D.tokens[begin + j]);
    };
    uint32_t key = n ? key_at(0) : D.V;
    bool head = key == before;
    int flags = 0;
    float acc[N];
    clear(acc);
    const auto keep = [&](int slot) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            sums[slot][threadIdx.x][i] = acc[i];
        if (lane == 0)
            key_of[slot][team] = key;
    };
    for (int j0 = 0; j0 < n && key < D.V; j0 += U) {
        uint32_t k[U];
        typename MemVec<VW>::type x[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            k[j] = j0 + j < n ? key_at(j0 + j) : D.V;
            if (k[j] < D.V)
                x[j] = load_vec<VW>(D.dout + uint64_t(row_at(j0 + j)) * D.row + off);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (j0 + j >= n)
                break;
            if (k[j] != key) {
                if (head) {
                    keep(0);
                    flags = HEAD;
                } else if (live) {
                    write_grad<G, ACC, N>(D, key, a, acc);
                }
                head = false;
                key = k[j];
                clear(acc);
            }
            if (key >= D.V)            // ignored ids come last
                break;
            float f[N];
            unpack<E, VW>(x[j], f);
            add(acc, f);
        }
    }
    if (key < D.V) {
        const bool on = key == after;
        if (head) {
            keep(0);
            flags = HEAD | (on ? ON : 0);
        } else if (on) {
            keep(1);
            flags |= TAIL;
        } else if (live) {
            write_grad<G, ACC, N>(D, key, a, acc);
        }
    }
    if (lane == 0)
        state[team] = flags;
    lds_barrier();
    const int merge = teams < kMerge ? teams : kMerge;
    if (team % merge != 0 || n == 0)
        return;
    const int64_t block = (int64_t{group} * teams + team) / merge;
    float *partial = D.partials + block * 2 * D.width + int64_t{a} * N;
    bool open = false;                  // a sum that goes on into the next team
    head = false;
    clear(acc);
    for (int t = team; t < team + merge; ++t) {
        const int s = state[t];
        const float(&h)[N] = sums[0][(t << lanes_log2) + lane], (&tail)[N] = sums[1][(t << lanes_log2) + lane];
        if (s & HEAD) {
            key = key_of[0][t];
            head = open ? head : true;
            open = s & ON;
            add(acc, h);
            if (!open) {
                if (live) {
                    if (head)
                        store_values<float, N>(reinterpret_cast<char *>(partial), acc);
                    else
                        write_grad<G, ACC, N>(D, key, a, acc);
                }
                head = false;
                clear(acc);
            }
        }
        if (s & TAIL) {
            clear(acc);
            add(acc, tail);
            open = true;
            head = false;
        }
    }
    if (open && live)
        store_values<float, N>(reinterpret_cast<char *>(head ? partial : partial + D.width), acc);
}

// The ids whose tokens lie in several blocks of chunk_sum_kernel: the work-
// group for the block in which an id begins adds its partial sums, each team of
// lanes a consecutive part of them, and then the teams' sums in order.  One id
// for 200000 tokens of 64 channels, 3125 partial sums, takes 29 us (128 with 64
// lanes a team, 8 of them at work, and the blocks found 64 at a time).
template <typename E, typename G, int VW, bool ACC>
__global__ __launch_bounds__(kSumThreads) void join_kernel(const GradDesc D)
{
    constexpr int N = VW / sizeof(E), U = 8;
    __shared__ float sums[kSumThreads][N];
    const int lanes = 1 << D.lanes_log2, lane = threadIdx.x & (lanes - 1);
    const int team = threadIdx.x >> D.lanes_log2, teams = kSumThreads >> D.lanes_log2;
    for (uint32_t block = blockIdx.x; block + 1 < D.blocks; block += gridDim.x) {
        const int64_t begin = block * D.block_tokens, end = begin + D.block_tokens;
        const uint32_t key = D.keys[end - 1];
        if (key >= D.V || D.keys[end] != key || (begin > 0 && D.keys[begin - 1] == key))
            continue;
        // the blocks with a part of it, this one and those whose first token
        // still has this id: of the next 64 in one look, then of all that are
        // left in 64 steps at a time
        int64_t n = 1, most = D.blocks - block;
        for (int64_t step = 1; n < most; step = (most - n + 63) / 64) {
            const int64_t i = n + ((threadIdx.x & 63) + 1) * step;
            const bool same = i <= most && D.keys[(block + i - 1) * D.block_tokens] == key;
            const int64_t found = __popcll(__ballot(same));
            if (found < 64 && n + (found + 1) * step - 1 < most)
                most = n + (found + 1) * step - 1;      // the first look that failed
            n += found * step;
        }
        const int64_t per = (n + teams - 1) / teams, i0 = team * per, i1 = i0 + per < n ? i0 + per : n;
        for (uint32_t a0 = blockIdx.y << D.lanes_log2; a0 < D.vecs; a0 += gridDim.y << D.lanes_log2) {
            const uint32_t a = a0 + lane;
            float acc[N];
            clear(acc);
            if (a < D.vecs) {
                const float *p = D.partials + int64_t{a} * N;
                for (int64_t i = i0; i < i1; i += U) {
                    float f[U][N];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        clear(f[u]);
                        if (i + u < i1)
                            load_values<float, N>(
                                reinterpret_cast<const char *>(p + ((block + i + u) * 2 + (i + u == 0)) * D.width),
                                f[u]);
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u)
                        add(acc, f[u]);
                }
            }
#pragma unroll
            for (int e = 0; e < N; ++e)
                sums[threadIdx.x][e] = acc[e];
            lds_barrier();
            if (team == 0 && a < D.vecs) {
                const int used = int((n + per - 1) / per);      // teams with a part
                for (int t = 1; t < used; ++t)
                    add(acc, sums[(t << D.lanes_log2) + lane]);
                write_grad<G, ACC, N>(D, key, a, acc);
            }
            lds_barrier();
        }
    }
}

// ------------------------------------------------------------- launches --

uint32_t groups_of(int64_t n, int64_t per) { return uint32_t((n + per - 1) / per); }

template <typename E, int VW>
const void *lookup_fn(bool uni)
{
    return uni ? reinterpret_cast<const void *>(lookup_kernel<E, VW, true>)
               : reinterpret_cast<const void *>(lookup_kernel<E, VW, false>);
}

struct GradFns {
    const void *sum, *join;
};

template <typename E, typename G, int VW, bool ACC>
GradFns grad_fns_of(bool uni)
{
    const void *join = reinterpret_cast<const void *>(join_kernel<E, G, VW, ACC>);
    if constexpr (VW == 16)            // narrower vectors are for rows of less than 16 bytes
        if (uni)
            return {reinterpret_cast<const void *>(chunk_sum_kernel<E, G, VW, true, ACC>), join};
    return {reinterpret_cast<const void *>(chunk_sum_kernel<E, G, VW, false, ACC>), join};
}

template <typename E, typename G, int VW>
GradFns grad_fns_of(bool uni, bool acc)
{
    return acc ? grad_fns_of<E, G, VW, true>(uni) : grad_fns_of<E, G, VW, false>(uni);
}

template <typename E, int VW>
GradFns grad_fns(basp_dtype grad, bool uni, bool acc)
{
    return grad == BASP_FP32   ? grad_fns_of<E, float, VW>(uni, acc)
           : grad == BASP_BF16 ? grad_fns_of<E, __bf16, VW>(uni, acc)
                               : grad_fns_of<E, _Float16, VW>(uni, acc);
}

basp_status launch_lookup(const basp_embed_plan &p, const void *ids, const void *table, float scale, void *out,
                          void *stream)
{
    const int vw = row_vector(p.D, p.es);
    const int64_t row = p.D * p.es, vecs = (row + vw - 1) / vw, step = std::max<int64_t>(1, kLaunchVectors / vecs);
    const void *fn = BASP_BY_ROW(lookup_fn, p.dtype, vw, vecs % 64 == 0);
    LookupDesc D = {};
    D.ids = ids;
    D.table = static_cast<const char *>(table);
    D.out = static_cast<char *>(out);
    D.V = p.V;
    D.row = uint32_t(row);
    D.per_row = make_fastdiv(uint32_t(vecs));
    D.order = p.order;
    D.scale = scale;
    D.wide_ids = p.id_bytes == 8;
    basp_status s = BASP_OK;
    for (int64_t t0 = 0; t0 < p.T && s == BASP_OK; t0 += step) {
        const int64_t n = std::min(step, p.T - t0);
        D.t0 = t0;
        D.nvec = n * vecs;
        s = launch_kernel(fn, dim3(groups_of(D.nvec, kThreads)), kThreads, D, stream, t0 == 0, t0 + n == p.T);
    }
    return s;
}

// Bytes of zeros beside the count and the place launch of a digit: about what
// HBM takes in the time of these launches with 32768 tokens and rows of 4 KiB.
// They follow neither tokens nor rows.  Whole gradients of 131072 rows with
// these, with half and with twice as many, and with none, us: 12001 tokens x 2048
// 103, 107, 103, 118; 32768 x 2048 123, 123, 124, 134; 262144 x 2048 355, 364,
// 353, 374; 32768 x 1024 79, 76, 85, 88; 32768 x 512 55, 52, 55, 61.
constexpr int64_t kBesideCount = int64_t{64} << 20, kBesidePlace = int64_t{160} << 20;

basp_status launch_grad(const basp_embed_plan &p, const void *ids, const void *dout, float scale, int accumulate,
                        void *dtable, void *ws, void *stream)
{
    char *const base = static_cast<char *>(ws);
    uint32_t *keys[2], *tokens[2];
    for (int i = 0; i < 2; ++i) {
        keys[i] = reinterpret_cast<uint32_t *>(base + p.keys[i]);
        tokens[i] = reinterpret_cast<uint32_t *>(base + p.tokens[i]);
    }
    ZeroDesc Z = {};
    Z.ids = ids;
    Z.tags = reinterpret_cast<uint32_t *>(base + p.tags);
    Z.dtable = static_cast<char *>(dtable);
    Z.T = p.T;
    Z.V = p.V;
    Z.padding = p.padding;
    Z.wide_ids = p.id_bytes == 8;

    basp_status s = BASP_OK;
    bool first = true;
    const auto go = [&](const void *fn, dim3 grid, int block, const auto &D, bool last, size_t lds) {
        if (s == BASP_OK)
            s = launch_kernel(fn, grid, block, D, stream, first, last, lds);
        first = false;
    };
    // Rows of the table are zeroed by the launches after the one that writes
    // the tags: as many beside the sort as its launches have time for, the
    // others beside the sums.
    const int64_t rows = accumulate ? 0 : p.V, row = p.D * p.grad_es;
    int64_t done = 0;
    const auto share = [&](int64_t bytes, int waves) {
        const int64_t end = std::min(rows, done + bytes / row);
        Z.z = zero_pieces(done, end, row, waves);
        done = end;
        return Z.z.groups;
    };
    if (p.T && p.sort_blocks == 0) {
        const RankDesc D = {keys[(p.passes - 1) & 1], tokens[(p.passes - 1) & 1], Z};
        const bool narrow = fits_narrow(p.T, p.V);
        go(narrow ? reinterpret_cast<const void *>(rank_kernel<uint32_t>)
                  : reinterpret_cast<const void *>(rank_kernel<uint64_t>),
           dim3(groups_of(p.T, kRankTokens)), kRankThreads, D, false,
           narrow ? rank_lds_bytes<uint32_t>(p.T) : rank_lds_bytes<uint64_t>(p.T));
    }
    for (int pass = 0; pass < p.passes && p.sort_blocks > 0 && p.T; ++pass) {
        PassDesc D = {};
        D.keys_in = keys[1 - (pass & 1)];
        D.tokens_in = tokens[1 - (pass & 1)];
        D.keys_out = keys[pass & 1];
        D.tokens_out = tokens[pass & 1];
        D.hist = reinterpret_cast<int32_t *>(base + p.hist);
        D.items = p.block_items;
        D.first = pass == 0;
        D.shift = pass * p.digit_bits;
        D.bins = 1 << p.digit_bits;
        D.groups = p.sort_blocks;
        const uint32_t with_count = share(pass == 0 ? 0 : kBesideCount, kSortWaves);
        D.zero = Z;
        go(reinterpret_cast<const void *>(digit_count_kernel), dim3(p.sort_blocks + with_count), kSortBlock, D, false,
           size_t(4) * D.bins);
        const uint32_t with_place = share(kBesidePlace, kSortWaves);
        D.zero = Z;
        go(p.block_items <= kSortItems       ? reinterpret_cast<const void *>(digit_place_kernel<kSortSteps>)
           : p.block_items <= 4 * kSortItems ? reinterpret_cast<const void *>(digit_place_kernel<4 * kSortSteps>)
                                             : reinterpret_cast<const void *>(digit_place_kernel<0>),
           dim3(p.sort_blocks + with_place), kSortBlock, D, false, sort_lds_bytes(kSortWaves, D.bins));
    }
    const int vw = row_vector(p.D, p.es), sorted = (p.passes - 1) & 1;
    const GradFns fn = BASP_BY_ROW(grad_fns, p.dtype, vw, p.grad_dtype, p.lanes_log2 == 6, accumulate != 0);
    GradDesc D = {};
    D.keys = keys[sorted];
    D.tokens = tokens[sorted];
    D.dout = static_cast<const char *>(dout);
    D.dtable = static_cast<char *>(dtable);
    D.partials = reinterpret_cast<float *>(base + p.partials);
    D.T = p.T;
    D.width = p.width;
    D.block_tokens = int64_t{p.chunk} * merged_teams(p.lanes_log2);
    D.V = uint32_t(p.V);
    D.blocks = uint32_t(p.blocks);
    D.row = uint32_t(p.D * p.es);
    D.grad_row = uint32_t(p.D * p.grad_es);
    D.elems = uint32_t(p.D);
    D.vecs = uint32_t((int64_t{D.row} + vw - 1) / vw);
    D.col_groups = make_fastdiv(uint32_t(p.col_groups));
    D.lanes_log2 = p.lanes_log2;
    D.chunk = p.chunk;
    D.sum_groups = uint32_t(p.sum_groups);
    D.order = p.order;
    D.scale = scale;
    const uint32_t zeros = share(INT64_MAX, kSumThreads / 64);
    D.zero = Z;
    const bool joins = p.blocks > 1;
    if (D.sum_groups + zeros)
        go(fn.sum, dim3(D.sum_groups + zeros), kSumThreads, D, !joins, 0);
    if (joins)
        go(fn.join, dim3(uint32_t(std::min<int64_t>(p.blocks - 1, 1 << 20)), std::min<uint32_t>(D.col_groups.d, 1024)),
           kSumThreads, D, true, 0);
    return s;
}

}  // namespace
}  // namespace basp

using basp::CallBuf;

extern "C" basp_status basp_embed_to_seq(const basp_embed_plan *p, const void *ids, const void *table, float scale,
                                         void *out, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p)
            return BASP_ERR_INVALID;
        const CallBuf in[] = {{ids, p->T * p->id_bytes, p->id_bytes}, {table, p->T ? p->V * p->D * p->es : 0, p->es}};
        const CallBuf o[] = {{out, p->T * p->D * p->es, p->es}};
        const basp_status s = basp::check_call(in, 2, o, 1);
        return s != BASP_OK ? s : basp::launch_lookup(*p, ids, table, scale, out, stream);
    });
}

extern "C" basp_status basp_embed_to_seq_grad(const basp_embed_plan *p, const void *ids, const void *dout,
                                              float scale, int accumulate, void *dtable, void *ws, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p)
            return BASP_ERR_INVALID;
        const CallBuf in[] = {{ids, p->T * p->id_bytes, p->id_bytes}, {dout, p->T * p->D * p->es, p->es}};
        const CallBuf o[] = {{dtable, p->V * p->D * p->grad_es, p->grad_es}, {ws, p->workspace_bytes, 16}};
        const basp_status s = basp::check_call(in, 2, o, 2);
        return s != BASP_OK ? s : basp::launch_grad(*p, ids, dout, scale, accumulate, dtable, ws, stream);
    });
}
