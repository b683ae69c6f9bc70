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
// partial sum and a count a work-group, and a second one joins them, or the only
// work-group does it itself.  Sums are fp32 in a fixed order, counts whole numbers.
// Scores of -infinity have no share and no gradient; rounding is to the scores'
// type at the end.
//
// Vector instructions bound it as much as reading does, so teams are small: 32768
// tokens x 320 in bf16 take 11 us in teams of 16 lanes with three vectors (21 MB),
// 13 us as a wave a token; the gradient 11 us, 15 us as a wave a token.  The join
// takes 7 us, a round of loads and an exchange between work-groups; one work-group
// needed 10 us for 256 x 320, at its rate of reading.  250 tokens x 8: 4 us.
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

// Partial results [groups][2][stride], the counts' last number the live tokens,
// and what becomes of them.
struct BalanceParts {
    float *parts, *shares;          // shares: of the loss, by the join's work-groups
    uint32_t *came;                 // those that are done
    float *loss, *slope;
    int32_t *counts;
    int32_t groups, E, K, stride;
    float coef;
};

struct BalanceDesc {
    const char *logits;
    const void *ids;
    const uint8_t *mask;
    int64_t T, per_group;           // tokens, and of a work-group
    uint32_t row, vecs;
    int32_t wide_ids;
    FastDiv by_K;
    BalanceParts out;
};

// The scores of a token in a team's registers: vector lane + r * LANES of the row,
// the last one of which may overlap the one before, or be beyond the row.
template <typename E, int VW, int LANES, int R>
struct Scores {
    static constexpr int N = VW / sizeof(E);
    typedef typename MemVec<VW>::type Raw;

    uint32_t lane, row, vecs, seen;         // seen: numbers of the last vector that the one before has
    bool has;                               // a last vector

    __device__ inline Scores(uint32_t lane_, uint32_t row_, uint32_t vecs_) : lane(lane_), row(row_), vecs(vecs_)
    {
        seen = first(R - 1);
        has = lane + (R - 1) * LANES < vecs;
    }
    __device__ inline uint32_t at(int r) const { return vec_offset<VW>(lane + r * LANES, row); }
    __device__ inline uint32_t first(int r) const { return ((lane + r * LANES) * VW - at(r)) / sizeof(E); }
    __device__ inline bool mine(int r, int i) const { return r < R - 1 || (has && uint32_t(i) >= seen); }

    __device__ inline void load(Raw (&x)[R], const char *row_at) const
    {
#pragma unroll
        for (int r = 0; r < R; ++r)         // beyond the row: its end, again
            x[r] = load_vec<VW, false>(row_at + at(r));
    }

    // exp(score - most) in f, 0 where another lane has the number; the return
    // value is their sum over the lane
    __device__ inline float powers(const Raw (&x)[R], float (&f)[R][N]) const
    {
        float most = -INFINITY;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            unpack<E, VW>(x[r], f[r]);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                f[r][i] = mine(r, i) ? f[r][i] : -INFINITY;
                most = fmaxf(most, f[r][i]);
            }
        }
        most = team_fold<LANES>(most, [](float a, float b) { return fmaxf(a, b); });
        float total = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                f[r][i] = __builtin_amdgcn_exp2f((f[r][i] - most) * 1.4426950408889634f);
                total += f[r][i];
            }
        return total;
    }
};

typedef float x4 __attribute__((ext_vector_type(4)));
typedef int i4 __attribute__((ext_vector_type(4)));

// Counts and slopes of the experts 4 c to 4 c + 3 from their sums and counts; their
// share of the loss.
__device__ inline float finish_experts(const BalanceParts &D, int c, int live, x4 P, i4 n)
{
    const float L = float(live);
    float term = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * c + i;
        if (e < D.E) {
            const float slope = live ? D.coef * (float(n[i]) * float(D.E) / (float(D.K) * L)) / L : 0.f;
            D.counts[e] = n[i];
            D.slope[e] = slope;
            term += live ? slope * P[i] : 0.f;
        }
    }
    return term;
}

template <typename E, int VW, int LANES, int R>
__global__ __launch_bounds__(kBalanceThreads) void balance_kernel(const BalanceDesc D)
{
    typedef Scores<E, VW, LANES, R> Row;
    constexpr int N = Row::N, TEAMS = kBalanceThreads / LANES, WAVES = kBalanceThreads / 64, WIDTH = R * LANES * N;
    __shared__ float part[WAVES][WIDTH];
    __shared__ __attribute__((aligned(16))) float total[kMaxExperts + 4];
    __shared__ __attribute__((aligned(16))) int hist[kMaxExperts + 4];
    const BalanceParts &out = D.out;
    const int64_t begin = blockIdx.x * D.per_group, end = begin + D.per_group < D.T ? begin + D.per_group : D.T;
    const Row row(threadIdx.x % LANES, D.row, D.vecs);
    // one token ahead; a masked token's scores are loaded too, and then ignored
    typename Row::Raw x[R];
    bool is = false;
    int64_t t = begin + threadIdx.x / LANES;
    if (t < end) {
        row.load(x, D.logits + t * D.row);
        is = !D.mask || D.mask[t];
    }
    for (int e = threadIdx.x; e < out.stride; e += kBalanceThreads) {
        hist[e] = 0;
        total[e] = 0.f;
    }
    lds_barrier();
    for (int64_t s = begin * out.K + threadIdx.x; s < end * out.K; s += kBalanceThreads) {
        const int64_t id = D.wide_ids ? static_cast<const int64_t *>(D.ids)[s] : static_cast<const int32_t *>(D.ids)[s];
        const bool live = !D.mask || D.mask[begin + fastdiv(uint32_t(s - begin * out.K), D.by_K)];
        if (live && id >= 0 && id < out.E)
            atomicAdd(&hist[id], 1);
    }
    float acc[R][N];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < N; ++i)
            acc[r][i] = 0.f;
    int live = 0;
    while (t < end) {
        typename Row::Raw now[R];
        const bool counts = is;
#pragma unroll
        for (int r = 0; r < R; ++r)
            now[r] = x[r];
        t += TEAMS;
        if (t < end) {
            row.load(x, D.logits + t * D.row);
            is = !D.mask || D.mask[t];
        }
        float f[R][N], sum[1] = {row.powers(now, f)};
        team_sum<LANES, 1>(sum, nullptr);
        const float inv = 1.f / sum[0];
        live += counts;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < N; ++i)
                acc[r][i] += counts ? f[r][i] * inv : 0.f;
    }
    if (row.lane == 0 && live)
        atomicAdd(&hist[out.E], live);
    // the teams' sums: those of a wave first, then the waves in their order
    const uint32_t wave = threadIdx.x >> 6;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            acc[r][i] = sum_of_teams<LANES>(acc[r][i]);
            if ((threadIdx.x & 63) < LANES)
                part[wave][(row.lane + r * LANES) * N + i] = acc[r][i];
        }
    lds_barrier();
    const bool alone = out.groups == 1;
    float *const parts = out.parts + int64_t(blockIdx.x) * 2 * out.stride, *const sums = alone ? total : parts;
    for (uint32_t c = threadIdx.x; c < WIDTH; c += kBalanceThreads) {
        const uint32_t a = c / N, off = vec_offset<VW>(a, D.row), seen = (a * VW - off) / sizeof(E);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            sum += part[w][c];
        if (a < D.vecs && c % N >= seen)
            sums[off / sizeof(E) + c % N] = sum;
    }
    if (!alone) {
        if (blockIdx.x == 0 && threadIdx.x == 0)
            *out.came = 0;          // for the next launch
        for (int e = threadIdx.x; e <= out.E; e += kBalanceThreads)
            reinterpret_cast<int *>(parts)[out.stride + e] = hist[e];
        return;
    }
    lds_barrier();
    const int c = threadIdx.x;
    float term = 0.f;
    if (4 * c < out.stride)
        term = finish_experts(out, c, hist[out.E], reinterpret_cast<const x4 *>(total)[c], reinterpret_cast<const i4 *>(hist)[c]);
    term = team_fold<64>(term, [](float a, float b) { return a + b; });
    if ((threadIdx.x & 63) == 0)
        part[wave][0] = term;
    lds_barrier();
    if (threadIdx.x == 0) {
        float loss = 0.f;
        for (int w = 0; w < WAVES; ++w)
            loss += part[w][0];
        *out.loss = loss;
    }
}

// kJoinColumns experts a work-group, four a thread, and 128 threads over the
// partial results.  The last work-group to come adds the shares of the loss, all in
// their order.
__global__ __launch_bounds__(kBalanceThreads) void balance_join_kernel(const BalanceParts D)
{
    constexpr int ACROSS = kJoinColumns / 4, SLICES = kBalanceThreads / ACROSS, WAVES = kBalanceThreads / 64, ROUNDS = kBalanceGroups / SLICES;
    __shared__ __attribute__((aligned(16))) x4 sums[WAVES][ACROSS];
    __shared__ __attribute__((aligned(16))) i4 counts[WAVES][ACROSS];
    __shared__ int live_tokens;
    const int fours = D.stride / 4, c = blockIdx.x * ACROSS + threadIdx.x % ACROSS, slice = threadIdx.x / ACROSS;
    if (threadIdx.x == 0)
        live_tokens = 0;
    const float *const from = D.parts + 4 * (c < fours ? c : 0);
    x4 x[ROUNDS];
    i4 y[ROUNDS];
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
        const int g = slice + i * SLICES < D.groups ? slice + i * SLICES : 0;
        x[i] = *reinterpret_cast<const x4 *>(from + int64_t{g} * 2 * D.stride);
        y[i] = *reinterpret_cast<const i4 *>(from + (int64_t{g} * 2 + 1) * D.stride);
    }
    lds_barrier();
    if (int(threadIdx.x) < D.groups)
        atomicAdd(&live_tokens, reinterpret_cast<const int *>(D.parts)[(int64_t{threadIdx.x} * 2 + 1) * D.stride + D.E]);
    x4 P = {0.f, 0.f, 0.f, 0.f};
    i4 n = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i)
        if (slice + i * SLICES < D.groups) {
            P += x[i];
            n += y[i];
        }
#pragma unroll
    for (int d = ACROSS; d < 64; d *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            P[i] += __shfl_xor(P[i], d);
            n[i] += __shfl_xor(n[i], d);
        }
    if ((threadIdx.x & 63) < ACROSS) {
        sums[threadIdx.x >> 6][threadIdx.x % ACROSS] = P;
        counts[threadIdx.x >> 6][threadIdx.x % ACROSS] = n;
    }
    lds_barrier();
    if (threadIdx.x >= 64)
        return;
    float term = 0.f;
    if (threadIdx.x < ACROSS && c < fours) {
        for (int w = 1; w < WAVES; ++w) {
            P += sums[w][threadIdx.x];
            n += counts[w][threadIdx.x];
        }
        term = finish_experts(D, c, live_tokens, P, n);
    }
    const auto add = [](float a, float b) { return a + b; };
    term = team_fold<64>(term, add);
    uint32_t came = 0;
    if (threadIdx.x == 0) {
        __hip_atomic_store(D.shares + blockIdx.x, term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        came = __hip_atomic_fetch_add(D.came, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (__builtin_amdgcn_readfirstlane(came) != gridDim.x - 1)
        return;
    float share = 0.f;              // gridDim.x is at most 33
    if (threadIdx.x < gridDim.x)
        share = __hip_atomic_load(D.shares + threadIdx.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    share = team_fold<64>(share, add);
    if (threadIdx.x == 0)
        *D.loss = share;
}

struct BalanceGradDesc {
    const char *logits;
    const uint8_t *mask;
    const float *slope, *dloss;
    char *dlogits;
    uint32_t tokens, row, vecs;
};

constexpr int kGradThreads = 256;

// Tokens of a team, one after the other, all on their way from the start.
constexpr int grad_tokens(int R) { return R <= 2 ? 4 : 2; }

template <typename E, int VW, int LANES, int R>
__global__ __launch_bounds__(kGradThreads) void balance_grad_kernel(const BalanceGradDesc D)
{
    typedef Scores<E, VW, LANES, R> Row;
    constexpr int N = Row::N, TEAMS = kGradThreads / LANES, U = grad_tokens(R);
    const uint32_t first = blockIdx.x * TEAMS * U + threadIdx.x / LANES;
    if (first >= D.tokens)
        return;
    const Row row(threadIdx.x % LANES, D.row, D.vecs);
    typename Row::Raw x[U][R];      // a masked token's, too, and then ignored
    bool live[U];
    float slope[R][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t t = first + u * TEAMS < D.tokens ? first + u * TEAMS : first;
        row.load(x[u], D.logits + uint64_t(t) * D.row);
        live[u] = !D.mask || D.mask[t];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
        load_values<float, N>(reinterpret_cast<const char *>(D.slope) + row.at(r) / sizeof(E) * 4, slope[r]);
    const float g = *D.dloss;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t t = first + u * TEAMS;
        float f[R][N], sums[2] = {row.powers(x[u], f), 0.f};
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < N; ++i)
                sums[1] += f[r][i] * slope[r][i];
        team_sum<LANES, 2>(sums, nullptr);
        const float inv = 1.f / sums[0], dot = sums[1] * inv, scale = g * inv;
        if (t >= D.tokens)
            return;
        char *const out = D.dlogits + uint64_t(t) * D.row;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float o[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                o[i] = live[u] ? scale * f[r][i] * (slope[r][i] - dot) : 0.f;
            if (r < R - 1 || (row.has && row.seen == 0))
                store_vec<VW>(out + row.at(r), pack<E, VW>(o));
            else
#pragma unroll
                for (int i = 0; i < N; ++i)     // the others belong to the lane before
                    if (row.mine(r, i))
                        reinterpret_cast<E *>(out + row.at(r))[i] = static_cast<E>(o[i]);
        }
    }
}

// --------------------------------------------------------------- launches --

struct BalanceShape {
    const void *sum, *grad;
    int tokens;                     // of a team of the gradient
};

template <typename E, int VW, int LANES, int R>
BalanceShape shape_of()
{
    return {reinterpret_cast<const void *>(balance_kernel<E, VW, LANES, R>),
            reinterpret_cast<const void *>(balance_grad_kernel<E, VW, LANES, R>), grad_tokens(R)};
}

template <typename E, int VW>
BalanceShape balance_shape(const LogitRow &r)
{
    if constexpr (VW == 16) {
        if (r.lanes == 8)
            return r.regs == 1   ? shape_of<E, VW, 8, 1>()
                   : r.regs == 2 ? shape_of<E, VW, 8, 2>()
                   : r.regs == 3 ? shape_of<E, VW, 8, 3>()
                                 : shape_of<E, VW, 8, 4>();
        if (r.lanes == 16)
            return r.regs == 3 ? shape_of<E, VW, 16, 3>() : shape_of<E, VW, 16, 4>();
        if (r.lanes == 32)
            return r.regs == 3 ? shape_of<E, VW, 32, 3>() : shape_of<E, VW, 32, 4>();
        if constexpr (kMaxExperts * sizeof(E) > 128 * VW)
            if (r.lanes == 64)
                return r.regs == 3 ? shape_of<E, VW, 64, 3>() : shape_of<E, VW, 64, 4>();
    }
    return shape_of<E, VW, 4, 1>();     // rows of shorter vectors have at most two
}

basp_status launch_balance(const basp_expert_plan &p, const void *logits, const void *ids, const uint8_t *mask, float coef,
                           float *loss, int32_t *counts, float *slope, void *ws, void *stream)
{
    const LogitRow r = logit_row(p);
    const BalanceShape shape = BASP_BY_ROW(balance_shape, p.weight_dtype, r.vw, r);
    const int groups = balance_groups(p);
    float *const parts = static_cast<float *>(ws);
    const int64_t partials = 2 * groups * balance_stride(p);
    const BalanceDesc D = {static_cast<const char *>(logits), ids, mask, p.T, (p.T + groups - 1) / groups, uint32_t(r.row),
                           uint32_t(r.vecs), p.id_bytes == 8, make_fastdiv(uint32_t(p.K)),
                           {parts, parts + partials + 1, reinterpret_cast<uint32_t *>(parts + partials), loss, slope, counts,
                            groups, p.E, p.K, int32_t(balance_stride(p)), coef}};
    basp_status s = launch_kernel(shape.sum, dim3(groups), kBalanceThreads, D, stream, true, groups == 1);
    if (s == BASP_OK && groups > 1)
        s = launch_kernel(reinterpret_cast<const void *>(balance_join_kernel), dim3(balance_joins(p)), kBalanceThreads,
                          D.out, stream, false, true);
    return s;
}

basp_status launch_balance_grad(const basp_expert_plan &p, const void *logits, const uint8_t *mask, const float *slope,
                                const float *dloss, void *dlogits, void *stream)
{
    const LogitRow r = logit_row(p);
    const BalanceShape shape = BASP_BY_ROW(balance_shape, p.weight_dtype, r.vw, r);
    const int64_t each = int64_t{kGradThreads / r.lanes} * shape.tokens, step = (int64_t{1} << 22) * each;
    basp_status s = BASP_OK;
    for (int64_t t0 = 0; t0 < p.T && s == BASP_OK; t0 += step) {
        const int64_t n = std::min(step, p.T - t0);
        const BalanceGradDesc D = {static_cast<const char *>(logits) + t0 * r.row, mask ? mask + t0 : nullptr, slope, dloss,
                                   static_cast<char *>(dlogits) + t0 * r.row, uint32_t(n), uint32_t(r.row), uint32_t(r.vecs)};
        s = launch_kernel(shape.grad, dim3(uint32_t((n + each - 1) / each)), kGradThreads, D, stream, t0 == 0, t0 + n == p.T);
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
        const int64_t need = int64_t(basp_balance_workspace_bytes(p));
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
