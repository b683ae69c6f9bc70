// balance.hip -- the balance loss of a router, its per-expert counts and its
// gradient: the kernels and entry points (basp.h, "Balance loss").
//
//   p = softmax(logits) per token,  P[e] = sum over live tokens of p[t][e],
//   f[e] = E counts[e] / (K L),  loss = coef sum_e f[e] P[e] / L
//   dlogits[t][j] = dloss p[t][j] (slope[j] - sum_e slope[e] p[t][e]),
//   slope = coef f / L
//
// A team of lanes holds a token's scores in registers, each lane the same
// columns of every token, and adds up the columns of p as it goes.  The scores
// are read once; small next to what a launch costs, so one launch makes a
// partial sum and a count a work-group, and one work-group joins them.  Sums
// are fp32 in a fixed order, counts whole numbers.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#define BASP_HD __host__ __device__
#include "layer_plan.hpp"
#include "plan_internal.hpp"
#include "rowvec.hpp"
#include "runtime.hpp"
#include "teams.hpp"

namespace basp {
namespace {

struct BalanceDesc {
    const char *logits;
    const void *ids;
    const uint8_t *mask;
    float *sums;                    // [groups][E]
    int32_t *counts;                // [groups][E + 1], the last: live tokens
    int64_t T, per_group;           // tokens, and of a work-group
    uint32_t row, vecs;
    int32_t K, E, wide_ids;
    FastDiv by_K;
};

// Scores of one token in a team's registers, -inf where a lane has no column
// of its own, and their softmax in place of them.
template <typename E, int VW, int LANES, int R>
struct Scores {
    static constexpr int N = VW / sizeof(E);
    float f[R][N];

    __device__ inline void load(const char *row_at, uint32_t lane, uint32_t row, uint32_t vecs)
    {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint32_t a = lane + r * LANES, off = vec_offset<VW>(a, row), seen = (a * VW - off) / sizeof(E);
            if (a < vecs)
                unpack<E, VW>(load_vec<VW, false>(row_at + off), f[r]);
#pragma unroll
            for (int i = 0; i < N; ++i)
                f[r][i] = a < vecs && uint32_t(i) >= seen ? f[r][i] : -INFINITY;
        }
    }

    __device__ inline void clear()
    {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < N; ++i)
                f[r][i] = 0.f;
    }

    __device__ inline void softmax()
    {
        float most = -INFINITY;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < N; ++i)
                most = fmaxf(most, f[r][i]);
        most = team_max<LANES>(most);
        float total[1] = {0.f};
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                f[r][i] = __builtin_amdgcn_exp2f((f[r][i] - most) * 1.4426950408889634f);
                total[0] += f[r][i];
            }
        team_sum<LANES, 1>(total, nullptr);
        const float inv = 1.f / total[0];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < N; ++i)
                f[r][i] *= inv;
    }
};

template <typename E, int VW, int LANES, int R>
__global__ __launch_bounds__(kBalanceThreads) void balance_kernel(const BalanceDesc D)
{
    constexpr int N = VW / sizeof(E), TEAMS = kBalanceThreads / LANES, WAVES = kBalanceThreads / 64;
    __shared__ float part[WAVES][(LANES < 64 ? LANES : 64) * N];
    __shared__ int hist[kMaxExperts + 1];
    const int64_t begin = blockIdx.x * D.per_group, end = begin + D.per_group < D.T ? begin + D.per_group : D.T;
    for (int e = threadIdx.x; e <= D.E; e += kBalanceThreads)
        hist[e] = 0;
    lds_barrier();
    const uint32_t lane = threadIdx.x % LANES;
    float acc[R][N];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < N; ++i)
            acc[r][i] = 0.f;
    int live = 0;
    // four tokens at a time: the sums over lanes of one are as long a chain as a
    // load from memory
    constexpr int U = 4;
    for (int64_t t = begin + threadIdx.x / LANES; t < end; t += TEAMS * U) {
        Scores<E, VW, LANES, R> s[U];
        bool is[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = t + u * TEAMS;
            if (at < end)               // a masked token's scores are loaded too, and then ignored
                s[u].load(D.logits + at * D.row, lane, D.row, D.vecs);
            else
                s[u].clear();
            is[u] = at < end && (!D.mask || D.mask[at]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u].softmax();
            live += is[u];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    acc[r][i] += is[u] ? s[u].f[r][i] : 0.f;
        }
    }
    if (lane == 0 && live)
        atomicAdd(&hist[D.E], live);
    for (int64_t s = begin * D.K + threadIdx.x; s < end * D.K; s += kBalanceThreads) {
        const int64_t id = D.wide_ids ? static_cast<const int64_t *>(D.ids)[s] : static_cast<const int32_t *>(D.ids)[s];
        if (id >= 0 && id < D.E && (!D.mask || D.mask[begin + fastdiv(uint32_t(s - begin * D.K), D.by_K)]))
            atomicAdd(&hist[id], 1);
    }
    // the teams' sums: those of a wave first, then the waves in their order
    const uint32_t wave = threadIdx.x >> 6, in_wave = threadIdx.x & 63;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int d = LANES; d < 64; d <<= 1)
                acc[r][i] += __shfl_xor(acc[r][i], d);
        lds_barrier();
        if (in_wave < LANES)
#pragma unroll
            for (int i = 0; i < N; ++i)
                part[wave][lane * N + i] = acc[r][i];
        lds_barrier();
        for (uint32_t c = threadIdx.x; c < LANES * N; c += kBalanceThreads) {
            const uint32_t a = c / N + r * LANES, off = vec_offset<VW>(a, D.row), seen = (a * VW - off) / sizeof(E);
            float sum = 0.f;
            for (int w = 0; w < WAVES; ++w)
                sum += part[w][c];
            if (a < D.vecs && c % N >= seen)
                D.sums[int64_t(blockIdx.x) * D.E + off / sizeof(E) + c % N] = sum;
        }
    }
    lds_barrier();
    for (int e = threadIdx.x; e <= D.E; e += kBalanceThreads)
        D.counts[int64_t(blockIdx.x) * (D.E + 1) + e] = hist[e];
}

struct BalanceJoinDesc {
    const float *sums;
    const int32_t *group_counts;
    float *loss, *slope;
    int32_t *counts;
    int32_t groups, E, K, columns_log2;
    float coef;
};

// One work-group: a power of two of columns side by side, and the rest of the
// threads over the partial sums.
__global__ __launch_bounds__(kBalanceThreads) void balance_join_kernel(const BalanceJoinDesc D)
{
    __shared__ float sums[kBalanceThreads];
    __shared__ int counts[kBalanceThreads];
    __shared__ float wave_loss[kBalanceThreads / 64];
    __shared__ int live_tokens;
    const int columns = 1 << D.columns_log2, e = threadIdx.x & (columns - 1), s = threadIdx.x >> D.columns_log2;
    const int slices = kBalanceThreads >> D.columns_log2;
    if (threadIdx.x == 0)
        live_tokens = 0;
    lds_barrier();
    float P = 0.f;
    int n = 0;
    if (e < D.E)
#pragma unroll 8
        for (int g = s; g < D.groups; g += slices) {
            P += D.sums[int64_t(g) * D.E + e];
            n += D.group_counts[int64_t(g) * (D.E + 1) + e];
        }
    for (int g = threadIdx.x; g < D.groups; g += kBalanceThreads)
        atomicAdd(&live_tokens, D.group_counts[int64_t(g) * (D.E + 1) + D.E]);
    sums[threadIdx.x] = P;
    counts[threadIdx.x] = n;
    lds_barrier();
    float term = 0.f;
    if (s == 0 && e < D.E) {
        for (int j = 1; j < slices; ++j) {
            P += sums[j * columns + e];
            n += counts[j * columns + e];
        }
        const float L = float(live_tokens);
        const float slope = live_tokens ? D.coef * (float(n) * float(D.E) / (float(D.K) * L)) / L : 0.f;
        D.counts[e] = n;
        D.slope[e] = slope;
        term = live_tokens ? slope * P : 0.f;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        term += __shfl_xor(term, d);
    if ((threadIdx.x & 63) == 0)
        wave_loss[threadIdx.x >> 6] = term;
    lds_barrier();
    if (threadIdx.x == 0) {
        float loss = 0.f;
        for (int w = 0; w < kBalanceThreads / 64; ++w)
            loss += wave_loss[w];
        *D.loss = loss;
    }
}

struct BalanceGradDesc {
    const char *logits;
    const uint8_t *mask;
    const float *slope, *dloss;
    char *dlogits;
    uint32_t tokens, row, vecs;
};

constexpr int kGradThreads = 256;

template <typename E, int VW, int LANES, int R>
__global__ __launch_bounds__(kGradThreads) void balance_grad_kernel(const BalanceGradDesc D)
{
    constexpr int N = VW / sizeof(E), TEAMS = kGradThreads / LANES;
    const uint32_t lane = threadIdx.x % LANES, t = blockIdx.x * TEAMS + threadIdx.x / LANES;
    if (t >= D.tokens)
        return;
    char *const out = D.dlogits + uint64_t(t) * D.row;
    Scores<E, VW, LANES, R> s;      // all loads first; a masked token's scores are then ignored
    float slope[R][N], dot[1] = {0.f};
    s.load(D.logits + uint64_t(t) * D.row, lane, D.row, D.vecs);
    const bool live = !D.mask || D.mask[t];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t a = lane + r * LANES;
#pragma unroll
        for (int i = 0; i < N; ++i)
            slope[r][i] = 0.f;
        if (a < D.vecs)
            load_values<float, N>(reinterpret_cast<const char *>(D.slope) + vec_offset<VW>(a, D.row) / sizeof(E) * 4, slope[r]);
    }
    const float g = *D.dloss;
    s.softmax();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < N; ++i)
            dot[0] += s.f[r][i] * slope[r][i];
    team_sum<LANES, 1>(dot, nullptr);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t a = lane + r * LANES, off = vec_offset<VW>(a, D.row), seen = (a * VW - off) / sizeof(E);
        float o[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            o[i] = live ? g * s.f[r][i] * (slope[r][i] - dot[0]) : 0.f;
        if (a < D.vecs) {
            if (seen == 0)
                store_vec<VW>(out + off, pack<E, VW>(o));
            else
#pragma unroll
                for (int i = 0; i < N; ++i)     // the others belong to the lane before
                    if (uint32_t(i) >= seen)
                        reinterpret_cast<E *>(out + off)[i] = static_cast<E>(o[i]);
        }
    }
}

// --------------------------------------------------------------- launches --

struct BalanceShape {
    const void *sum, *grad;
    int lanes;
};

template <typename E, int VW, int LANES, int R>
BalanceShape shape_of()
{
    return {reinterpret_cast<const void *>(balance_kernel<E, VW, LANES, R>),
            reinterpret_cast<const void *>(balance_grad_kernel<E, VW, LANES, R>), LANES};
}

// As many lanes as a token has vectors, so that few are idle; at most a wave.
template <typename E, int VW>
BalanceShape balance_shape(int64_t vecs)
{
    if (vecs <= 4)
        return shape_of<E, VW, 4, 1>();
    if constexpr (VW == 16) {
        if (vecs <= 16)
            return shape_of<E, VW, 16, 1>();
        if (vecs <= 32)
            return shape_of<E, VW, 32, 1>();
        if (vecs <= 64)
            return shape_of<E, VW, 64, 1>();
        if (vecs <= 128)
            return shape_of<E, VW, 64, 2>();
        return shape_of<E, VW, 64, 4>();
    }
    return {};                       // shorter vectors: a row holds at most two
}

struct LogitRow {
    int vw;
    int64_t row, vecs;
};

LogitRow logit_row(const basp_expert_plan &p)
{
    LogitRow r;
    r.vw = row_vector(p.E, p.ws_es);
    r.row = int64_t{p.E} * p.ws_es;
    r.vecs = (r.row + r.vw - 1) / r.vw;
    return r;
}

basp_status launch_balance(const basp_expert_plan &p, const void *logits, const void *ids, const uint8_t *mask, float coef,
                           float *loss, int32_t *counts, float *slope, void *ws, void *stream)
{
    const LogitRow r = logit_row(p);
    const BalanceShape shape = BASP_BY_ROW(balance_shape, p.weight_dtype, r.vw, r.vecs);
    const int groups = p.T ? balance_groups(p) : 0;
    float *const sums = static_cast<float *>(ws);
    int32_t *const group_counts = reinterpret_cast<int32_t *>(sums + int64_t{groups} * p.E);
    const BalanceDesc D = {static_cast<const char *>(logits), ids, mask, sums, group_counts, p.T,
                           groups ? (p.T + groups - 1) / groups : 0, uint32_t(r.row), uint32_t(r.vecs), p.K, p.E,
                           p.id_bytes == 8, make_fastdiv(uint32_t(p.K))};
    basp_status s = BASP_OK;
    if (groups)
        s = launch_kernel(shape.sum, dim3(groups), kBalanceThreads, D, stream, true, false);
    BalanceJoinDesc J = {sums, group_counts, loss, slope, counts, groups, p.E, p.K, 0, coef};
    while ((1 << J.columns_log2) < p.E)
        ++J.columns_log2;
    if (s == BASP_OK)
        s = launch_kernel(reinterpret_cast<const void *>(balance_join_kernel), dim3(1), kBalanceThreads, J, stream, !groups, true);
    return s;
}

basp_status launch_balance_grad(const basp_expert_plan &p, const void *logits, const uint8_t *mask, const float *slope,
                                const float *dloss, void *dlogits, void *stream)
{
    const LogitRow r = logit_row(p);
    const BalanceShape shape = BASP_BY_ROW(balance_shape, p.weight_dtype, r.vw, r.vecs);
    const int64_t teams = kGradThreads / shape.lanes, step = (int64_t{1} << 22) * teams;
    basp_status s = BASP_OK;
    for (int64_t t0 = 0; t0 < p.T && s == BASP_OK; t0 += step) {
        const int64_t n = std::min(step, p.T - t0);
        const BalanceGradDesc D = {static_cast<const char *>(logits) + t0 * r.row, mask ? mask + t0 : nullptr, slope, dloss,
                                   static_cast<char *>(dlogits) + t0 * r.row, uint32_t(n), uint32_t(r.row), uint32_t(r.vecs)};
        s = launch_kernel(shape.grad, dim3(uint32_t((n + teams - 1) / teams)), kGradThreads, D, stream, t0 == 0, t0 + n == p.T);
    }
    return s;
}

}  // namespace
}  // namespace basp

using basp::CallBuf;

extern "C" basp_status basp_balance_loss(const basp_expert_plan *p, const void *logits, const void *ids, const uint8_t *mask,
                                         float coef, float *loss, int32_t *counts, float *slope, void *ws, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p || !std::isfinite(coef))
            return BASP_ERR_INVALID;
        const CallBuf in[] = {{logits, p->T * p->E * p->ws_es, p->ws_es}, {ids, p->slots * p->id_bytes, p->id_bytes},
                              {mask, mask ? p->T : 0, 1}};
        const int64_t need = int64_t{basp::balance_groups(*p)} * (2 * p->E + 1) * 4;
        const CallBuf out[] = {{loss, 4, 4}, {counts, int64_t{4} * p->E, 4}, {slope, int64_t{4} * p->E, 4}, {ws, need, 16}};
        const basp_status s = basp::check_call(in, 3, out, 4);
        return s != BASP_OK ? s : basp::launch_balance(*p, logits, ids, mask, coef, loss, counts, slope, ws, stream);
    });
}

extern "C" basp_status basp_balance_loss_grad(const basp_expert_plan *p, const void *logits, const uint8_t *mask,
                                              const float *slope, const float *dloss, void *dlogits, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p)
            return BASP_ERR_INVALID;
        const int64_t n = p->T * p->E * p->ws_es;
        const CallBuf in[] = {{logits, n, p->ws_es}, {mask, mask ? p->T : 0, 1}, {slope, int64_t{4} * p->E, 4}, {dloss, 4, 4}};
        const CallBuf out[] = {{dlogits, n, p->ws_es}};
        const basp_status s = basp::check_call(in, 4, out, 1);
        return s != BASP_OK ? s : basp::launch_balance_grad(*p, logits, mask, slope, dloss, dlogits, stream);
    });
}
