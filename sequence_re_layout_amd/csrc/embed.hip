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
// to the token's place.  UNI: a row is a whole number of waves.
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

// ------------------------------------------------------- tokens by their id --

// One pass of the sort by id, least significant digit first.
struct PassDesc {
    const void *ids;                // first pass: ids as given
    const uint32_t *keys_in, *tokens_in;
    uint32_t *keys_out, *tokens_out;
    int32_t *hist;
    int64_t T, items, V, padding;
    int32_t first, wide_ids, shift, bins;
};

__device__ inline uint32_t pass_key(const PassDesc &D, int64_t i)
{
    return D.first ? row_of_id(D.ids, i, D.V, D.padding, D.wide_ids) : D.keys_in[i];
}

__global__ __launch_bounds__(kSortBlock) void digit_count_kernel(const PassDesc D)
{
    extern __shared__ int lds[];
    const int64_t begin = blockIdx.x * D.items, end = begin + D.items < D.T ? begin + D.items : D.T;
    sort_count<kSortWaves>(lds, begin, end, D.bins, D.hist + int64_t{blockIdx.x} * D.bins,
                           [&](int64_t i) { return int(pass_key(D, i) >> D.shift) & (D.bins - 1); });
}

__global__ __launch_bounds__(kSortBlock) void digit_place_kernel(const PassDesc D)
{
    extern __shared__ int lds[];
    const int64_t begin = blockIdx.x * D.items, end = begin + D.items < D.T ? begin + D.items : D.T;
    sort_place<kSortWaves>(
        sort_lds(lds, kSortWaves, D.bins), begin, end, D.bins, 1, D.hist, gridDim.x, blockIdx.x,
        [&](int64_t i) { return int(pass_key(D, i) >> D.shift) & (D.bins - 1); },
        [&](int64_t i, int, int at) {
            if (at < D.T) {
                D.keys_out[at] = pass_key(D, i);
                D.tokens_out[at] = D.first ? uint32_t(i) : D.tokens_in[i];
            }
        });
}

// ------------------------------------------------------- sums by their id --

struct GradDesc {
    const uint32_t *keys, *tokens;  // sorted
    const char *dout;
    char *dtable;
    float *partials;                // [chunks][2][width]
    int64_t T, width;
    uint32_t V, chunks, row, vecs, grad_row, elems;
    FastDiv col_groups;             // column groups of a chunk: vecs / lanes, rounded up
    int32_t lanes_log2;             // lanes of a column group
    int64_t items;                  // chunks * column groups
    uint32_t sum_groups;            // work-groups that sum; the others write zeros
    basp_seq_order order;
    float scale;
    int32_t accumulate;
};

// The channels of vector a of table row `key`, scaled, as they are written.
template <typename G, int N>
__device__ inline void write_grad(const GradDesc &D, uint32_t key, uint32_t a, const float (&sum)[N])
{
    const uint32_t first = a * N, last = D.elems - N, at = first < last ? first : last;
    char *p = D.dtable + uint64_t(key) * D.grad_row + uint64_t(at) * sizeof(G);
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = sum[i] * D.scale;
    if (D.accumulate) {
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

// Rows of the table that no token names, as zeros: 64 rows a work-group.
template <typename G>
__device__ inline void zero_unnamed(const GradDesc &D, uint32_t group, uint32_t groups)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (uint32_t r0 = group * 64; r0 < D.V; r0 += groups * 64) {
        const uint32_t r = r0 + lane;
        // the first sorted key that is not below r
        int64_t lo = 0, hi = D.T;
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (D.keys[mid] < r)
                lo = mid + 1;
            else
                hi = mid;
        }
        uint64_t m = __ballot(r < D.V && (lo == D.T || D.keys[lo] != r));
        for (int n = 0; m; ++n, m &= m - 1)
            if (n % (kThreads / 64) == wave)
                zero_row(D.dtable + uint64_t(r0 + __builtin_ctzll(m)) * D.grad_row, D.grad_row, lane);
    }
}

// The sorted tokens in chunks of kChunk: a lane sums one vector of channels
// over its chunk and writes the sum wherever the id changes.  An id whose
// tokens lie in several chunks leaves one fp32 partial sum per chunk: slot 0
// where it began in an earlier chunk, slot 1 where it begins in this one.
template <typename E, typename G, int VW>
__global__ __launch_bounds__(kThreads) void chunk_sum_kernel(const GradDesc D)
{
    constexpr int N = VW / sizeof(E), U = 8;
    if (blockIdx.x >= D.sum_groups) {
        zero_unnamed<G>(D, blockIdx.x - D.sum_groups, gridDim.x - D.sum_groups);
        return;
    }
    const uint32_t lanes = 1u << D.lanes_log2;
    const int64_t item = int64_t{blockIdx.x} * (kThreads >> D.lanes_log2) + (threadIdx.x >> D.lanes_log2);
    if (item >= D.items)
        return;
    const uint32_t chunk = fastdiv(uint32_t(item), D.col_groups);
    const uint32_t a = (uint32_t(item) - chunk * D.col_groups.d) * lanes + (threadIdx.x & (lanes - 1));
    if (a >= D.vecs)
        return;
    const uint32_t off = vec_offset<VW>(a, D.row);
    const int64_t begin = int64_t{chunk} * kChunk, end = begin + kChunk < D.T ? begin + kChunk : D.T;
    float *partial = D.partials + int64_t{chunk} * 2 * D.width + int64_t{a} * N;

    uint32_t key = D.keys[begin];
    bool began_before = begin > 0 && D.keys[begin - 1] == key;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        acc[i] = 0.f;
    for (int64_t i0 = begin; i0 < end && key < D.V; i0 += U) {
        uint32_t k[U];
        typename MemVec<VW>::type x[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            k[j] = i0 + j < end ? D.keys[i0 + j] : D.V;
            if (k[j] < D.V)
                x[j] = load_vec<VW>(D.dout + uint64_t(seq_row(D.order, D.tokens[i0 + j])) * D.row + off);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (i0 + j >= end)
                break;
            if (k[j] != key) {
                if (began_before)
                    store_values<float, N>(reinterpret_cast<char *>(partial), acc);
                else
                    write_grad<G, N>(D, key, a, acc);
                began_before = false;
                key = k[j];
#pragma unroll
                for (int i = 0; i < N; ++i)
                    acc[i] = 0.f;
            }
            if (key >= D.V)            // ignored ids come last
                break;
            float f[N];
            unpack<E, VW>(x[j], f);
#pragma unroll
            for (int i = 0; i < N; ++i)
                acc[i] += f[i];
        }
    }
    if (key >= D.V)
        return;
    const bool goes_on = end < D.T && D.keys[end] == key;
    if (began_before)
        store_values<float, N>(reinterpret_cast<char *>(partial), acc);
    else if (goes_on)
        store_values<float, N>(reinterpret_cast<char *>(partial + D.width), acc);
    else
        write_grad<G, N>(D, key, a, acc);
}

// The ids whose tokens lie in several chunks: the work-group of the chunk in
// which one begins adds its partial sums, each wave a consecutive part of
// them and then the waves' sums in order.
constexpr int kJoinWaves = 8;

template <typename E, typename G, int VW>
__global__ __launch_bounds__(64 * kJoinWaves) void join_kernel(const GradDesc D)
{
    constexpr int N = VW / sizeof(E);
    __shared__ float sums[kJoinWaves][64][N];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (uint32_t chunk = blockIdx.x; chunk + 1 < D.chunks; chunk += gridDim.x) {
        const int64_t begin = int64_t{chunk} * kChunk, end = begin + kChunk;
        const uint32_t key = D.keys[end - 1];
        if (key >= D.V || D.keys[end] != key || (begin > 0 && D.keys[begin - 1] == key))
            continue;
        // past the last token with this key
        int64_t lo = end, hi = D.T;
        while (lo < hi) {
            const int64_t mid = (lo + hi) >> 1;
            if (D.keys[mid] <= key)
                lo = mid + 1;
            else
                hi = mid;
        }
        const int64_t last = (lo - 1) / kChunk, n = last - chunk + 1;   // chunks with a part of it
        const int64_t per = (n + kJoinWaves - 1) / kJoinWaves, i0 = wave * per, i1 = i0 + per < n ? i0 + per : n;
        for (uint32_t a0 = blockIdx.y * 64; a0 < D.vecs; a0 += gridDim.y * 64) {
            const uint32_t a = a0 + lane;
            float acc[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                acc[i] = 0.f;
            if (a < D.vecs) {
                const float *p = D.partials + int64_t{a} * N;
#pragma unroll 4
                for (int64_t i = i0; i < i1; ++i) {
                    float f[N];
                    load_values<float, N>(
                        reinterpret_cast<const char *>(p + ((chunk + i) * 2 + (i == 0)) * D.width), f);
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        acc[e] += f[e];
                }
            }
#pragma unroll
            for (int e = 0; e < N; ++e)
                sums[wave][lane][e] = acc[e];
            __syncthreads();
            if (wave == 0 && a < D.vecs) {
                for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        acc[e] += sums[w][lane][e];
                write_grad<G, N>(D, key, a, acc);
            }
            __syncthreads();
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

template <typename E, int VW>
GradFns grad_fns(basp_dtype grad)
{
    if (grad == BASP_FP32)
        return {reinterpret_cast<const void *>(chunk_sum_kernel<E, float, VW>),
                reinterpret_cast<const void *>(join_kernel<E, float, VW>)};
    if (grad == BASP_BF16)
        return {reinterpret_cast<const void *>(chunk_sum_kernel<E, __bf16, VW>),
                reinterpret_cast<const void *>(join_kernel<E, __bf16, VW>)};
    return {reinterpret_cast<const void *>(chunk_sum_kernel<E, _Float16, VW>),
            reinterpret_cast<const void *>(join_kernel<E, _Float16, VW>)};
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

basp_status launch_grad(const basp_embed_plan &p, const void *ids, const void *dout, float scale, int accumulate,
                        void *dtable, void *ws, void *stream)
{
    char *const base = static_cast<char *>(ws);
    uint32_t *keys[2], *tokens[2];
    for (int i = 0; i < 2; ++i) {
        keys[i] = reinterpret_cast<uint32_t *>(base + p.keys[i]);
        tokens[i] = reinterpret_cast<uint32_t *>(base + p.tokens[i]);
    }
    basp_status s = BASP_OK;
    bool first = true;
    const auto go = [&](const void *fn, dim3 grid, int block, const auto &D, bool last, size_t lds) {
        if (s == BASP_OK)
            s = launch_kernel(fn, grid, block, D, stream, first, last, lds);
        first = false;
    };
    int from = 1;                       // the pass before wrote keys[from]
    for (int pass = 0; pass < p.passes && p.T; ++pass) {
        PassDesc D = {};
        D.ids = ids;
        D.keys_in = keys[from];
        D.tokens_in = tokens[from];
        D.keys_out = keys[1 - from];
        D.tokens_out = tokens[1 - from];
        D.hist = reinterpret_cast<int32_t *>(base + p.hist);
        D.T = p.T;
        D.items = p.block_items;
        D.V = p.V;
        D.padding = p.padding;
        D.first = pass == 0;
        D.wide_ids = p.id_bytes == 8;
        D.shift = pass * p.digit_bits;
        D.bins = 1 << p.digit_bits;
        if (p.sort_blocks > 1)
            go(reinterpret_cast<const void *>(digit_count_kernel), dim3(p.sort_blocks), kSortBlock, D, false,
               size_t(4) * D.bins);
        go(reinterpret_cast<const void *>(digit_place_kernel), dim3(p.sort_blocks), kSortBlock, D, false,
           sort_lds_bytes(kSortWaves, D.bins));
        from = 1 - from;
    }
    const int vw = row_vector(p.D, p.es);
    const GradFns fn = BASP_BY_ROW(grad_fns, p.dtype, vw, p.grad_dtype);
    GradDesc D = {};
    D.keys = keys[from];
    D.tokens = tokens[from];
    D.dout = static_cast<const char *>(dout);
    D.dtable = static_cast<char *>(dtable);
    D.partials = reinterpret_cast<float *>(base + p.partials);
    D.T = p.T;
    D.width = p.width;
    D.V = uint32_t(p.V);
    D.chunks = uint32_t(p.chunks);
    D.row = uint32_t(p.D * p.es);
    D.grad_row = uint32_t(p.D * p.grad_es);
    D.elems = uint32_t(p.D);
    D.vecs = uint32_t((int64_t{D.row} + vw - 1) / vw);
    while (D.lanes_log2 < 6 && (1u << D.lanes_log2) < D.vecs)
        ++D.lanes_log2;
    const uint32_t col_groups = groups_of(D.vecs, 1 << D.lanes_log2);
    D.col_groups = make_fastdiv(col_groups);
    D.items = p.chunks * col_groups;
    D.sum_groups = groups_of(D.items, kThreads >> D.lanes_log2);
    D.order = p.order;
    D.scale = scale;
    D.accumulate = accumulate != 0;
    const uint32_t zeros = accumulate ? 0 : uint32_t(std::min<int64_t>(1 << 20, (p.V + 63) / 64));
    const bool joins = p.chunks > 1;
    if (D.sum_groups + zeros)
        go(fn.sum, dim3(D.sum_groups + zeros), kThreads, D, !joins, 0);
    if (joins)
        go(fn.join, dim3(uint32_t(std::min<int64_t>(p.chunks - 1, 1 << 20)), std::min<uint32_t>(groups_of(D.vecs, 64), 1024)), 64 * kJoinWaves, D,
           true, 0);
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
