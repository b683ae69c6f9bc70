// expert.hip -- tokens sorted by expert and back: the kernels and entry points
// of the expert plans (basp.h, "Index-driven re-layouts").
//
// Every kernel but the sort moves rows of D channels and is bound by HBM: a
// lane holds one 16-byte vector of a row, so that each row is read once and
// written once, and the sums and products ride along in fp32 registers.
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
constexpr int64_t kLaunchVectors = int64_t{1} << 30;   // vectors of one launch: 31-bit division, 32-bit grid

struct SortDesc {
    const void *ids;
    int32_t *pos, *order, *offsets, *counts;
    int32_t *hist;
    int64_t slots, items;           // items: slots of one work-group
    int32_t E, align, max_rows, wide_ids;
};

__device__ inline int expert_of(const void *ids, int64_t i, int E, int wide)
{
    const int64_t id = wide ? static_cast<const int64_t *>(ids)[i] : static_cast<const int32_t *>(ids)[i];
    return id >= 0 && id < E ? int(id) : -1;
}

__global__ __launch_bounds__(kSortBlock) void expert_count_kernel(const SortDesc D)
{
    extern __shared__ int lds[];
    const int64_t begin = blockIdx.x * D.items, end = begin + D.items < D.slots ? begin + D.items : D.slots;
    sort_count<kSortWaves>(lds, begin, end, D.E, D.hist + int64_t{blockIdx.x} * D.E,
                           [&](int64_t i) { return expert_of(D.ids, i, D.E, D.wide_ids); });
}

// Ranks and places the slots.  Bound by latency: two rounds of loads, the
// matches and a scan (131072 slots of 64 experts: 5.9 us, and 4.8 for the
// counts before).  R: 64-item steps of a wave whose experts stay in registers,
// or 0 (sort.hpp).
template <int R>
__global__ __launch_bounds__(kSortBlock) void expert_place_kernel(const SortDesc D)
{
    extern __shared__ int lds[];
    const SortLds l = sort_lds(lds, kSortWaves, D.E);
    const int group = blockIdx.x, groups = gridDim.x, tid = threadIdx.x;
    const int64_t begin = group * D.items, end = begin + D.items < D.slots ? begin + D.items : D.slots;
    sort_place<kSortWaves, R>(
        l, begin, end, D.E, D.align, D.hist, groups, group,
        [&](int64_t i) { return expert_of(D.ids, i, D.E, D.wide_ids); }, [](int e) { return e; },
        [&](int64_t i, int, int at) {
            D.pos[i] = at;
            if (at >= 0 && at < D.max_rows)
                D.order[at] = int32_t(i);
        });
    // rows without a slot: the padding of this group's share of the experts, an
    // expert to a wave, and the group's share of what lies behind the last one
    if (D.align > 1)
        for (int e = group * kSortWaves + (tid >> 6); e < D.E; e += groups * kSortWaves)
            for (int64_t r = int64_t{l.start[e]} + l.total[e] + (tid & 63); r < l.start[e + 1]; r += 64)
                D.order[r] = -1;
    for (int64_t r = l.start[D.E] + int64_t{group} * kSortBlock + tid; r < D.max_rows; r += int64_t{groups} * kSortBlock)
        D.order[r] = -1;
    if (group == 0) {
        for (int e = tid; e < D.E; e += kSortBlock)
            D.counts[e] = l.total[e];
        for (int e = tid; e <= D.E; e += kSortBlock)
            D.offsets[e] = l.start[e];
    }
}

// Rows without a slot are few as a rule: work-groups of their own look
// through `order`, up to 64 rows in one go, and share out what they find.
struct ZeroDesc {
    char *out;
    const int32_t *order;
    uint32_t max_rows, slots, row;
    uint32_t look, groups;          // rows in one go, work-groups
};

constexpr int64_t kZeroGroups = 1 << 20;

__device__ inline void zero_unnamed(const ZeroDesc &D, uint32_t group)
{
    constexpr int WAVES = kThreads / 64;
    const int lane = threadIdx.x & 63, wave = scalar(threadIdx.x >> 6);
    for (uint32_t r0 = group * D.look; r0 < D.max_rows; r0 += D.groups * D.look) {
        const uint32_t r = r0 + lane;
        uint64_t m = __ballot(uint32_t(lane) < D.look && r < D.max_rows && uint32_t(D.order[r]) >= D.slots);
        for (int n = 0; m; ++n, m &= m - 1)
            if (n % WAVES == wave)
                zero_span(D.out + uint64_t(r0 + __builtin_ctzll(m)) * D.row, D.row, lane, 64);
    }
}

// Rows of `row` bytes in vectors of VW bytes, `per_row` of them each.
struct MoveDesc {
    const char *x;
    char *out;
    const int32_t *pos;
    int64_t nvec;                   // vectors of the tokens of this launch
    uint32_t row;
    FastDiv per_row;
    int32_t K;
    uint32_t max_rows;
    uint32_t move_groups;           // work-groups of the tokens; the others write zeros
    ZeroDesc zero;
};

// seq -> expert: each lane reads one vector of a token and writes it to the
// rows of the token's slots.  UNI: a row is a whole number of waves, so the
// token is the same for a wave and its index comes through scalar loads.  Bound
// by HBM writes to many places at once: 32768 tokens x 2048, 4 slots each, 706
// MB in 130 us (5.4 TB/s), as bare stores in this pattern (5.3-5.4).  Tokens
// gathered by row instead are read K times: 155 us.
template <int VW, bool UNI>
__global__ __launch_bounds__(kThreads) void scatter_kernel(const MoveDesc D)
{
    if (blockIdx.x >= D.move_groups) {
        zero_unnamed(D.zero, blockIdx.x - D.move_groups);
        return;
    }
    const uint32_t v = blockIdx.x * kThreads + threadIdx.x;
    if (v >= D.nvec)
        return;
    uint32_t t = fastdiv(v, D.per_row);
    if constexpr (UNI)
        t = scalar(t);
    const uint32_t off = vec_offset<VW>(v - t * D.per_row.d, D.row);
    const auto x = load_vec<VW, false>(D.x + uint64_t(t) * D.row + off);
    const int32_t *pos = D.pos + uint64_t(t) * D.K;
    for (int k = 0; k < D.K; ++k) {
        const uint32_t p = pos[k];
        if (p < D.max_rows)
            store_vec<VW>(D.out + uint64_t(p) * D.row + off, x);
    }
}

// The sort and the move of a small call in one launch: every work-group ranks
// all the slots, keeps those of its own rows, and copies these rows.  Up to
// kRouteSlots slots this is faster than three launches (1200 slots of 4 KiB:
// 7.7 against 12.4 us, 2048: 11.7 against 13.0; with 4096 it would be 20.5
// against 13.2).
constexpr int kRouteWaves = kThreads / 64, kRouteSteps = 8;
constexpr int kRouteSlots = kThreads * kRouteSteps;
constexpr int kRouteRows = 64;      // rows of a work-group at most
constexpr int64_t kRouteGroups = 1024;

struct RouteDesc {
    SortDesc sort;
    const char *x;
    char *out;
    uint32_t row;
    FastDiv per_row, K;
    int32_t rows;                   // of a work-group
};

template <int VW>
__global__ __launch_bounds__(kThreads) void route_kernel(const RouteDesc D)
{
    extern __shared__ int lds[];
    __shared__ int slot_of[kRouteRows];
    const SortDesc &S = D.sort;
    const SortLds l = sort_lds(lds, kRouteWaves, S.E);
    const int tid = threadIdx.x, first = blockIdx.x * D.rows;
    const int rows = first + D.rows < S.max_rows ? D.rows : S.max_rows - first;
    if (tid < kRouteRows)
        slot_of[tid] = -1;
    sort_place<kRouteWaves, kRouteSteps>(
        l, 0, S.slots, S.E, S.align, nullptr, 1, 0,
        [&](int64_t i) { return expert_of(S.ids, i, S.E, S.wide_ids); }, [](int e) { return e; },
        [&](int64_t i, int, int at) {
            if (blockIdx.x == 0)
                S.pos[i] = at;
            if (at >= first && at < first + rows)
                slot_of[at - first] = int(i);
        });
    lds_barrier();
    if (blockIdx.x == 0) {
        for (int e = tid; e < S.E; e += kThreads)
            S.counts[e] = l.total[e];
        for (int e = tid; e <= S.E; e += kThreads)
            S.offsets[e] = l.start[e];
    }
    if (tid < rows)
        S.order[first + tid] = slot_of[tid];
    const uint32_t n = rows * D.per_row.d;
    for (uint32_t v = tid; v < n; v += kThreads) {
        const uint32_t r = fastdiv(v, D.per_row), off = vec_offset<VW>(v - r * D.per_row.d, D.row);
        const int slot = slot_of[r];
        typename MemVec<VW>::type x = {};
        if (slot >= 0)
            x = load_vec<VW, false>(D.x + uint64_t(fastdiv(slot, D.K)) * D.row + off);
        store_vec<VW, false>(D.out + uint64_t(first + r) * D.row + off, x);
    }
}

struct SumDesc {
    const char *rows;
    char *out;
    const int32_t *pos;
    const void *weights;            // at the launch's first slot
    int64_t nvec;
    uint32_t row;
    FastDiv per_row;
    int32_t K;
    uint32_t max_rows;
    basp_dtype weight_dtype;
    int32_t streamed;               // store past the XCD's caches
};

// Sums of at least this many bytes are stored past the XCD's caches.  Weighted
// sums in bf16 with such stores and without, us (2048 channels, 4 choices; 4096,
// 2; 512, 8): 16 MiB 15.7 / 15.7, 10.0 / 9.8, 26.7 / 26.3; 32 MiB 29.2 / 28.8,
// 18.3 / 18.2, 51.0 / 50.3; 64 MiB 57.0 / 57.3, 34.9 / 34.9, 100.7 / 100.2; 96
// MiB 83.7 / 85.8, 49.4 / 49.8, 150.3 / 150.7; 128 MiB 111.4 / 113.6, 66.0 /
// 67.1, 201.6 / 203.0.  They gain from about 64 MiB on and cost up to 2%
// between 32 and 64; the smallest calls end later (16 tokens x 4096, 8 choices:
// 5.4 against 4.5).
constexpr int64_t kStreamBytes = int64_t{32} << 20;

// expert -> seq and the gradient of seq -> expert: out[t] = sum over k of
// (weights[t][k] *) rows[pos[t][k]] in fp32, k ascending.  KB loads are in
// flight at a time; dropped slots are not read.  Bound by HBM: 32768 x 4096, 2
// slots, 806 MB in 126 us (6.4 TB/s, 95% of a copy); 32768 x 2048, 4 slots, 672
// MB in 111 us.
template <typename E, int VW, int KB, bool WEIGHTED, bool UNI>
__global__ __launch_bounds__(kThreads) void gather_sum_kernel(const SumDesc D)
{
    constexpr int N = VW / sizeof(E);
    const uint32_t v = blockIdx.x * kThreads + threadIdx.x;
    if (v >= D.nvec)
        return;
    uint32_t t = fastdiv(v, D.per_row);
    if constexpr (UNI)
        t = scalar(t);
    const uint32_t off = vec_offset<VW>(v - t * D.per_row.d, D.row);
    const uint64_t slot = uint64_t(t) * D.K;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        acc[i] = 0.f;
    for (int k0 = 0; k0 < D.K; k0 += KB) {
        uint32_t p[KB];
        float w[KB];
        typename MemVec<VW>::type x[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const bool in = k0 + j < D.K;
            p[j] = in ? uint32_t(D.pos[slot + k0 + j]) : 0xffffffffu;
            if constexpr (WEIGHTED)
                w[j] = in ? load_number(D.weights, slot + k0 + j, D.weight_dtype) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < KB; ++j)
            if (p[j] < D.max_rows)
                x[j] = load_vec<VW>(D.rows + uint64_t(p[j]) * D.row + off);
#pragma unroll
        for (int j = 0; j < KB; ++j)
            if (p[j] < D.max_rows) {
                float f[N];
                unpack<E, VW>(x[j], f);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    acc[i] = WEIGHTED ? fmaf(w[j], f[i], acc[i]) : acc[i] + f[i];
            }
    }
    char *const out = D.out + uint64_t(t) * D.row;
    if constexpr (UNI && VW == 16) {
        if (D.streamed) {
            store_streamed(out, D.row, off, pack<E, VW>(acc));
            return;
        }
    }
    store_vec<VW>(out + off, pack<E, VW>(acc));
}

struct GradDesc {
    const char *dout, *rows;
    char *drows;
    const int32_t *pos;
    const void *weights;
    void *dweights;
    uint32_t tokens, row, vecs;
    int32_t K, lanes_log2;          // lanes that share a token: 8 to 256
    uint32_t max_rows;
    uint32_t token_groups;          // work-groups of the tokens; the others write zeros
    basp_dtype weight_dtype;
    ZeroDesc zero;
};

// The sums of KB values over `span` lanes (a power of two, at least KB), one
// of them to a lane: lane l gets that of value summed_by<KB>(l).  Half of the
// values go to the other lane of a pair in each of the first steps, so that
// a wave sums 8 values in 10 exchanges instead of 48.
template <int KB>
__device__ inline int summed_by(int lane)
{
    int j = 0;
#pragma unroll
    for (int b = 1; b < KB; b <<= 1)
        j = j << 1 | ((lane & b) != 0);
    return j;
}

template <int KB>
__device__ inline float sum_over_lanes(float (&v)[KB], int lane, int span)
{
#pragma unroll
    for (int b = 1; b < KB; b <<= 1) {
        const bool upper = lane & b;
        const int half = KB / (2 * b);
#pragma unroll
        for (int i = 0; i < half; ++i) {
            const float keep = upper ? v[i + half] : v[i], send = upper ? v[i] : v[i + half];
            v[i] = keep + __shfl_xor(send, b);
        }
    }
    float sum = v[0];
#pragma unroll
    for (int d = KB; d < 64; d <<= 1)
        if (d < span)
            sum += __shfl_xor(sum, d);
    return sum;
}

// The gradient of expert -> seq.  2^lanes_log2 lanes (8 up to the whole work-
// group) take a token: each reads its vectors of dout, and per slot reads the
// row's vector, adds the product to the slot's dot product and writes the
// weighted dout.  The dot products are then summed over the lanes.
// UNI: a token takes whole waves, so that its index and weights are scalars.
// Bound by HBM where there are many tokens: 16384 x 2048, 8 slots, 1143 MB in
// 206 us (5.5 TB/s).  The bare reads and writes of this pattern take 208 us, and
// 217 with non-temporal reads of dout, which may come from the Infinity Cache.
// By one work-group's chain of loads, sums and stores where there are few.
template <typename E, int VW, int KB, bool UNI>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(const GradDesc D)
{
    constexpr int N = VW / sizeof(E), WAVES = kThreads / 64;
    __shared__ float part[2][WAVES][KB];
    if (blockIdx.x >= D.token_groups) {
        zero_unnamed(D.zero, blockIdx.x - D.token_groups);
        return;
    }
    const uint32_t lanes = 1u << D.lanes_log2, lane = threadIdx.x & (lanes - 1);
    uint32_t t = blockIdx.x * (kThreads >> D.lanes_log2) + (threadIdx.x >> D.lanes_log2);
    if constexpr (UNI)
        t = scalar(t);
    const bool live = t < D.tokens;
    const uint64_t slot = uint64_t(t) * D.K;
    const char *dout = D.dout + uint64_t(t) * D.row;
    for (int k0 = 0; k0 < D.K; k0 += KB) {
        uint32_t p[KB];
        float w[KB], dot[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            const bool in = live && k0 + j < D.K;
            p[j] = in ? uint32_t(D.pos[slot + k0 + j]) : 0xffffffffu;
            w[j] = in ? load_number(D.weights, slot + k0 + j, D.weight_dtype) : 0.f;
            dot[j] = 0.f;
        }
        for (uint32_t a = lane; live && a < D.vecs; a += lanes) {
            const uint32_t off = vec_offset<VW>(a, D.row);
            const uint32_t seen = (a * VW - off) / sizeof(E);   // elements the vector before holds too
            float g[N];
            unpack<E, VW>(load_vec<VW, false>(dout + off), g);
            typename MemVec<VW>::type x[KB];
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (p[j] < D.max_rows)
                    x[j] = load_vec<VW>(D.rows + uint64_t(p[j]) * D.row + off);
#pragma unroll
            for (int j = 0; j < KB; ++j)
                if (p[j] < D.max_rows) {
                    float f[N], y[N];
                    unpack<E, VW>(x[j], f);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        dot[j] = uint32_t(i) < seen ? dot[j] : fmaf(g[i], f[i], dot[j]);
                        y[i] = w[j] * g[i];
                    }
                    store_vec<VW>(D.drows + uint64_t(p[j]) * D.row + off, pack<E, VW>(y));
                }
        }
        const int wave = threadIdx.x >> 6, l = threadIdx.x & 63, j = summed_by<KB>(l);
        float sum = sum_over_lanes<KB>(dot, l, lanes < 64 ? lanes : 64);
        if (lanes > 64) {
            // batches use the two halves of `part` in turn: the barrier of the
            // next one lies between a read here and the write after it
            float(&mine)[WAVES][KB] = part[k0 / KB & 1];
            if (l < KB)
                mine[wave][j] = sum;
            lds_barrier();
            if (lane < KB) {
                sum = mine[wave][j];
                for (uint32_t i = 1; i < lanes >> 6; ++i)
                    sum += mine[wave + i][j];
            }
        }
        if (lane < KB && live && k0 + j < D.K)
            store_number(D.dweights, slot + k0 + j, D.weight_dtype, sum);
    }
}

// ------------------------------------------------------------- launches --

SortDesc sort_desc(const basp_expert_plan &p, const void *ids, int32_t *pos, int32_t *order, int32_t *offsets,
                   int32_t *counts, void *ws)
{
    return {ids, pos, order, offsets, counts, static_cast<int32_t *>(ws), p.slots, p.block_items,
            p.E, p.align, int32_t(p.max_rows), p.id_bytes == 8};
}

basp_status launch_sort(const basp_expert_plan &p, const SortDesc &D, void *stream, bool last)
{
    const dim3 grid(p.sort_blocks);
    const void *place =
        p.block_items <= kSortItems       ? reinterpret_cast<const void *>(expert_place_kernel<kSortSteps>)
        : p.block_items <= 4 * kSortItems ? reinterpret_cast<const void *>(expert_place_kernel<4 * kSortSteps>)
                                          : reinterpret_cast<const void *>(expert_place_kernel<0>);
    basp_status s = BASP_OK;
    if (p.sort_blocks > 1)
        s = launch_kernel(reinterpret_cast<const void *>(expert_count_kernel), grid, kSortBlock, D, stream, true, false,
                          size_t(4) * p.E);
    if (s == BASP_OK)
        s = launch_kernel(place, grid, kSortBlock, D, stream, p.sort_blocks == 1, last,
                          sort_lds_bytes(kSortWaves, p.E));
    return s;
}

// f(token0, tokens, first, last) for launches of at most kLaunchVectors
// vectors each.
template <typename F>
basp_status by_launch(int64_t T, int64_t per_row, F f)
{
    const int64_t step = std::max<int64_t>(1, kLaunchVectors / per_row);
    basp_status s = BASP_OK;
    for (int64_t t = 0; t < T && s == BASP_OK; t += step)
        s = f(t, std::min(step, T - t), t == 0, t + step >= T);
    return s;
}

uint32_t groups_of(int64_t n, int64_t per) { return uint32_t((n + per - 1) / per); }

struct RowShape {
    int vw;
    int64_t row, vecs;
};

RowShape row_shape(const basp_expert_plan &p)
{
    RowShape r;
    r.vw = row_vector(p.D, p.es);
    r.row = p.D * p.es;
    r.vecs = (r.row + r.vw - 1) / r.vw;
    return r;
}

ZeroDesc zero_desc(const basp_expert_plan &p, int64_t row, const int32_t *order, void *out)
{
    // one row a wave while that does not fill the device
    const int64_t look = std::min<int64_t>(64, std::max<int64_t>(kThreads / 64, p.max_rows / 1024));
    return {static_cast<char *>(out), order, uint32_t(p.max_rows), uint32_t(p.slots), uint32_t(row), uint32_t(look),
            uint32_t(std::min(kZeroGroups, (p.max_rows + look - 1) / look))};
}

template <int VW>
const void *scatter_fn(bool uni)
{
    return uni ? reinterpret_cast<const void *>(scatter_kernel<VW, true>)
               : reinterpret_cast<const void *>(scatter_kernel<VW, false>);
}

template <typename E, int VW, int KB>
const void *sum_fn(bool weighted, bool uni)
{
    if (weighted)
        return uni ? reinterpret_cast<const void *>(gather_sum_kernel<E, VW, KB, true, true>)
                   : reinterpret_cast<const void *>(gather_sum_kernel<E, VW, KB, true, false>);
    return uni ? reinterpret_cast<const void *>(gather_sum_kernel<E, VW, KB, false, true>)
               : reinterpret_cast<const void *>(gather_sum_kernel<E, VW, KB, false, false>);
}

template <typename E, int VW>
const void *sum_fn(int K, bool weighted, bool uni)
{
    return K == 1   ? sum_fn<E, VW, 1>(weighted, uni)
           : K == 2 ? sum_fn<E, VW, 2>(weighted, uni)
           : K <= 4 ? sum_fn<E, VW, 4>(weighted, uni)
                    : sum_fn<E, VW, 8>(weighted, uni);
}

// Slots of a token that are in flight at a time: up to 8, or 4 in fp32 (4092
// tokens of 777 channels, 5 choices: 29.5 us with 4, 33.4 with 8; 16384 tokens
// of 2048 in bf16, 8 choices: 208 with 4, 205 with 8).
template <typename E, int VW, bool UNI>
const void *grad_fn_of(int K)
{
    constexpr int MOST = sizeof(E) == 4 ? 4 : 8;
    return K == 1   ? reinterpret_cast<const void *>(combine_grad_kernel<E, VW, 1, UNI>)
           : K == 2 ? reinterpret_cast<const void *>(combine_grad_kernel<E, VW, 2, UNI>)
           : K <= 4 ? reinterpret_cast<const void *>(combine_grad_kernel<E, VW, 4, UNI>)
                    : reinterpret_cast<const void *>(combine_grad_kernel<E, VW, MOST, UNI>);
}

template <typename E, int VW>
const void *grad_fn(int K, bool uni)
{
    return uni ? grad_fn_of<E, VW, true>(K) : grad_fn_of<E, VW, false>(K);
}

template <int VW>
const void *route_fn()
{
    return reinterpret_cast<const void *>(route_kernel<VW>);
}

// Whether a call is one launch of route_kernel.
bool route_in_one(const basp_expert_plan &p, const RowShape &r)
{
    return p.slots <= kRouteSlots && p.max_rows > 0 && p.max_rows <= kRouteGroups * kRouteRows &&
           p.max_rows * r.vecs <= kLaunchVectors;
}

basp_status launch_route(const basp_expert_plan &p, const RowShape &r, const SortDesc &S, const void *x, void *out,
                         void *stream)
{
    const void *fn = r.vw == 16  ? route_fn<16>()
                     : r.vw == 8 ? route_fn<8>()
                     : r.vw == 4 ? route_fn<4>()
                                 : route_fn<2>();
    RouteDesc D = {};
    D.sort = S;
    D.x = static_cast<const char *>(x);
    D.out = static_cast<char *>(out);
    D.row = uint32_t(r.row);
    D.per_row = make_fastdiv(uint32_t(r.vecs));
    D.K = make_fastdiv(uint32_t(p.K));
    D.rows = int32_t((p.max_rows + kRouteGroups - 1) / kRouteGroups);
    return launch_kernel(fn, dim3(groups_of(p.max_rows, D.rows)), kThreads, D, stream, true, true,
                         sort_lds_bytes(kRouteWaves, p.E));
}

basp_status launch_scatter(const basp_expert_plan &p, const void *x, const int32_t *pos, const int32_t *order,
                           void *out, void *stream, bool first_call)
{
    const RowShape r = row_shape(p);
    const bool uni = r.vecs % 64 == 0;
    const void *fn = r.vw == 16  ? scatter_fn<16>(uni)
                     : r.vw == 8 ? scatter_fn<8>(uni)
                     : r.vw == 4 ? scatter_fn<4>(uni)
                                 : scatter_fn<2>(uni);
    return by_launch(p.T, r.vecs, [&](int64_t t0, int64_t n, bool first, bool last) {
        MoveDesc D = {};
        D.x = static_cast<const char *>(x) + t0 * r.row;
        D.out = static_cast<char *>(out);
        D.pos = pos + t0 * p.K;
        D.nvec = n * r.vecs;
        D.row = uint32_t(r.row);
        D.per_row = make_fastdiv(uint32_t(r.vecs));
        D.K = p.K;
        D.max_rows = uint32_t(p.max_rows);
        D.zero = zero_desc(p, r.row, order, out);
        D.move_groups = groups_of(D.nvec, kThreads);
        const uint32_t zeros = last ? D.zero.groups : 0;
        return launch_kernel(fn, dim3(D.move_groups + zeros), kThreads, D, stream, first && first_call, last);
    });
}

basp_status launch_sum(const basp_expert_plan &p, const void *rows, const int32_t *pos, const void *weights, void *out,
                       void *stream)
{
    const RowShape r = row_shape(p);
    const void *fn = BASP_BY_ROW(sum_fn, p.dtype, r.vw, p.K, weights != nullptr, r.vecs % 64 == 0);
    return by_launch(p.T, r.vecs, [&](int64_t t0, int64_t n, bool first, bool last) {
        SumDesc D = {};
        D.rows = static_cast<const char *>(rows);
        D.out = static_cast<char *>(out) + t0 * r.row;
        D.pos = pos + t0 * p.K;
        D.weights = weights ? static_cast<const char *>(weights) + t0 * p.K * p.ws_es : nullptr;
        D.nvec = n * r.vecs;
        D.row = uint32_t(r.row);
        D.per_row = make_fastdiv(uint32_t(r.vecs));
        D.K = p.K;
        D.max_rows = uint32_t(p.max_rows);
        D.weight_dtype = p.weight_dtype;
        D.streamed = p.T * r.row >= kStreamBytes;
        return launch_kernel(fn, dim3(groups_of(D.nvec, kThreads)), kThreads, D, stream, first, last);
    });
}

basp_status launch_grad(const basp_expert_plan &p, const void *dout, const void *rows, const int32_t *pos,
                        const int32_t *order, const void *weights, void *drows, void *dweights, void *stream)
{
    const RowShape r = row_shape(p);
    GradDesc D = {};
    D.row = uint32_t(r.row);
    D.vecs = uint32_t(r.vecs);
    D.K = p.K;
    D.max_rows = uint32_t(p.max_rows);
    D.zero = zero_desc(p, r.row, order, drows);
    D.weight_dtype = p.weight_dtype;
    D.rows = static_cast<const char *>(rows);
    D.drows = static_cast<char *>(drows);
    D.lanes_log2 = 3;
    while (D.lanes_log2 < 8 && (int64_t{1} << D.lanes_log2) < r.vecs)
        ++D.lanes_log2;
    const void *fn = BASP_BY_ROW(grad_fn, p.dtype, r.vw, p.K, D.lanes_log2 >= 6);
    const int64_t per_group = kThreads >> D.lanes_log2, step = (int64_t{1} << 22) * per_group;
    basp_status s = BASP_OK;
    for (int64_t t0 = 0; t0 < p.T && s == BASP_OK; t0 += step) {
        const int64_t n = std::min(step, p.T - t0);
        const bool last = t0 + n == p.T;
        D.dout = static_cast<const char *>(dout) + t0 * r.row;
        D.pos = pos + t0 * p.K;
        D.weights = static_cast<const char *>(weights) + t0 * p.K * p.ws_es;
        D.dweights = static_cast<char *>(dweights) + t0 * p.K * p.ws_es;
        D.tokens = uint32_t(n);
        D.token_groups = groups_of(n, per_group);
        const uint32_t zeros = last ? D.zero.groups : 0;
        s = launch_kernel(fn, dim3(D.token_groups + zeros), kThreads, D, stream, t0 == 0, last);
    }
    return s;
}

// ------------------------------------------------------------- the checks --

struct ExpertBytes {
    int64_t x, rows, pos, order, offsets, counts, ids, weights;
};

ExpertBytes bytes_of(const basp_expert_plan &p)
{
    return {p.T * p.D * p.es, p.max_rows * p.D * p.es, p.slots * 4, p.max_rows * 4, (int64_t{p.E} + 1) * 4,
            int64_t{p.E} * 4, p.slots * p.id_bytes, p.slots * p.ws_es};
}

}  // namespace
}  // namespace basp

using basp::CallBuf;

extern "C" basp_status basp_expert_sort(const basp_expert_plan *p, const void *ids, int32_t *pos, int32_t *order,
                                        int32_t *offsets, int32_t *counts, void *ws, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p)
            return BASP_ERR_INVALID;
        const basp::ExpertBytes n = basp::bytes_of(*p);
        const CallBuf in[] = {{ids, n.ids, p->id_bytes}};
        const CallBuf out[] = {{pos, n.pos, 4}, {order, n.order, 4}, {offsets, n.offsets, 4}, {counts, n.counts, 4},
                               {ws, p->workspace_bytes, 16}};
        const basp_status s = basp::check_call(in, 1, out, 5);
        return s != BASP_OK ? s : basp::launch_sort(*p, basp::sort_desc(*p, ids, pos, order, offsets, counts, ws), stream, true);
    });
}

extern "C" basp_status basp_seq_to_expert(const basp_expert_plan *p, const void *x, const int32_t *pos,
                                          const int32_t *order, void *out, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p)
            return BASP_ERR_INVALID;
        const basp::ExpertBytes n = basp::bytes_of(*p);
        const CallBuf in[] = {{x, n.x, p->es}, {pos, n.pos, 4}, {order, n.order, 4}};
        const CallBuf o[] = {{out, n.rows, p->es}};
        const basp_status s = basp::check_call(in, 3, o, 1);
        return s != BASP_OK ? s : basp::launch_scatter(*p, x, pos, order, out, stream, true);
    });
}

extern "C" basp_status basp_route_to_expert(const basp_expert_plan *p, const void *x, const void *ids, int32_t *pos,
                                            int32_t *order, int32_t *offsets, int32_t *counts, void *out, void *ws,
                                            void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p)
            return BASP_ERR_INVALID;
        const basp::ExpertBytes n = basp::bytes_of(*p);
        const CallBuf in[] = {{x, n.x, p->es}, {ids, n.ids, p->id_bytes}};
        const CallBuf o[] = {{pos, n.pos, 4}, {order, n.order, 4}, {offsets, n.offsets, 4}, {counts, n.counts, 4},
                             {out, n.rows, p->es}, {ws, p->workspace_bytes, 16}};
        basp_status s = basp::check_call(in, 2, o, 6);
        if (s != BASP_OK)
            return s;
        const basp::SortDesc D = basp::sort_desc(*p, ids, pos, order, offsets, counts, ws);
        const basp::RowShape r = basp::row_shape(*p);
        if (basp::route_in_one(*p, r))
            return basp::launch_route(*p, r, D, x, out, stream);
        s = basp::launch_sort(*p, D, stream, p->T == 0);
        return s != BASP_OK ? s : basp::launch_scatter(*p, x, pos, order, out, stream, false);
    });
}

extern "C" basp_status basp_seq_to_expert_grad(const basp_expert_plan *p, const void *dout, const int32_t *pos,
                                               void *dx, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p)
            return BASP_ERR_INVALID;
        const basp::ExpertBytes n = basp::bytes_of(*p);
        const CallBuf in[] = {{dout, n.rows, p->es}, {pos, n.pos, 4}};
        const CallBuf o[] = {{dx, n.x, p->es}};
        const basp_status s = basp::check_call(in, 2, o, 1);
        return s != BASP_OK ? s : basp::launch_sum(*p, dout, pos, nullptr, dx, stream);
    });
}

extern "C" basp_status basp_expert_to_seq(const basp_expert_plan *p, const void *rows, const int32_t *pos,
                                          const void *weights, void *out, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p)
            return BASP_ERR_INVALID;
        const basp::ExpertBytes n = basp::bytes_of(*p);
        const CallBuf in[] = {{rows, n.rows, p->es}, {pos, n.pos, 4}, {weights, n.weights, p->ws_es}};
        const CallBuf o[] = {{out, n.x, p->es}};
        const basp_status s = basp::check_call(in, 3, o, 1);
        return s != BASP_OK ? s : basp::launch_sum(*p, rows, pos, weights, out, stream);
    });
}

extern "C" basp_status basp_expert_to_seq_grad(const basp_expert_plan *p, const void *dout, const void *rows,
                                               const int32_t *pos, const int32_t *order, const void *weights,
                                               void *drows, void *dweights, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p)
            return BASP_ERR_INVALID;
        const basp::ExpertBytes n = basp::bytes_of(*p);
        const CallBuf in[] = {{dout, n.x, p->es}, {rows, n.rows, p->es}, {pos, n.pos, 4}, {order, n.order, 4},
                              {weights, n.weights, p->ws_es}};
        const CallBuf o[] = {{drows, n.rows, p->es}, {dweights, n.weights, p->ws_es}};
        const basp_status s = basp::check_call(in, 5, o, 2);
        return s != BASP_OK ? s : basp::launch_grad(*p, dout, rows, pos, order, weights, drows, dweights, stream);
    });
}
