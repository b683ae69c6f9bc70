// norm.hip -- layer norm of token rows and its gradients: the kernels and entry
// points of the norm plans (basp.h, "Layer norm").
//
// Bound by HBM: a row is read once into registers, its mean and the sum of
// squares about that mean are taken there in fp32 (two passes over registers,
// so that a mean far from zero costs no digits), and it is written once.  The
// gradient reads the row and its gradient once; the weight's and the bias's
// gradients ride along in registers over the rows of a work-group, which leaves
// one partial sum of each, and a second launch adds these in a fixed order.
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

constexpr int kThreads = 256;
constexpr int64_t kLaunchGroups = int64_t{1} << 22;     // work-groups of one launch: 32-bit global size

struct NormDesc {
    const char *x;
    const void *weight, *bias;
    char *y;
    float *mean, *rstd;
    uint32_t rows, row, vecs, D;    // row: bytes
    float eps, inv_D;
    basp_dtype weight_dtype;
};

// Elements at the front of vector a that the vector before it holds too.
template <typename E, int VW>
__device__ inline uint32_t shared_front(uint32_t a, uint32_t off)
{
    return (a * VW - off) / sizeof(E);
}

template <typename E, int VW>
__device__ inline void norm_vector(typename MemVec<VW>::type x, float mean, float rstd, const float (&w)[VW / sizeof(E)],
                                   const float (&b)[VW / sizeof(E)], char *y)
{
    constexpr int N = VW / sizeof(E);
    float f[N];
    unpack<E, VW>(x, f);
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = fmaf((f[i] - mean) * rstd, w[i], b[i]);
    store_vec<VW>(y, pack<E, VW>(f));
}

// The weight and the bias of a vector's channels.
template <typename E, int VW>
__device__ inline void load_weights(const NormDesc &D, uint32_t off, float (&w)[VW / sizeof(E)], float (&b)[VW / sizeof(E)])
{
    constexpr int N = VW / sizeof(E);
    load_any<N>(D.weight, off / sizeof(E), D.weight_dtype, w);
#pragma unroll
    for (int i = 0; i < N; ++i)
        b[i] = 0.f;
    if (D.bias)
        load_any<N>(D.bias, off / sizeof(E), D.weight_dtype, b);
}

// LANES lanes take a row, R vectors each, and keep the weights of their channels
// in registers over the rows that they take in turn; the next row is on its way
// while one is normed.  32768 rows of 4096 in bf16: 95 to 98 us, 5.5 TB/s; with
// weights read anew for each row 298 us.  16 rows: 3.5 us.
template <typename E, int VW, int LANES, int R>
__global__ __launch_bounds__(LANES > kThreads ? LANES : kThreads) void norm_kernel(const NormDesc D)
{
    constexpr int N = VW / sizeof(E), TEAMS = LANES > kThreads ? 1 : kThreads / LANES;
    __shared__ float lds[2][LANES > 64 ? LANES / 64 : 1];
    const uint32_t lane = threadIdx.x % LANES, team = threadIdx.x / LANES, step = gridDim.x * TEAMS;
    uint32_t off[R], seen[R];
    float w[R][N], b[R][N];
    typename MemVec<VW>::type v[R];
    const auto fetch = [&](uint32_t t) {
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (t < D.rows && lane + r * LANES < D.vecs)
                v[r] = load_vec<VW, true>(D.x + uint64_t(t) * D.row + off[r]);
    };
#pragma unroll
    for (int r = 0; r < R; ++r) {
        off[r] = vec_offset<VW>(lane + r * LANES, D.row);
        seen[r] = lane + r * LANES < D.vecs ? shared_front<E, VW>(lane + r * LANES, off[r]) : N;
    }
    fetch(blockIdx.x * TEAMS + team);
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (lane + r * LANES < D.vecs)
            load_weights<E, VW>(D, off[r], w[r], b[r]);
    for (uint32_t first = blockIdx.x * TEAMS; first < D.rows; first += step) {
        const uint32_t t = first + team;
        typename MemVec<VW>::type x[R];
        float sum[1] = {0.f}, sq[1] = {0.f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            x[r] = v[r];
            float f[N];
            unpack<E, VW>(x[r], f);
#pragma unroll
            for (int i = 0; i < N; ++i)
                sum[0] += uint32_t(i) < seen[r] ? 0.f : f[i];
        }
        fetch(t + step);
        team_sum<LANES, 1>(sum, lds[0]);
        const float mean = sum[0] * D.inv_D;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float f[N];
            unpack<E, VW>(x[r], f);
#pragma unroll
            for (int i = 0; i < N; ++i)
                sq[0] += uint32_t(i) < seen[r] ? 0.f : (f[i] - mean) * (f[i] - mean);
        }
        team_sum<LANES, 1>(sq, lds[1]);
        const float rstd = 1.f / sqrtf(sq[0] * D.inv_D + D.eps);
        if (t >= D.rows)
            continue;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (lane + r * LANES < D.vecs)
                norm_vector<E, VW>(x[r], mean, rstd, w[r], b[r], D.y + uint64_t(t) * D.row + off[r]);
        if (lane == 0) {
            if (D.mean)
                D.mean[t] = mean;
            if (D.rstd)
                D.rstd[t] = rstd;
        }
    }
}

// Rows of more vectors than the registers of a work-group hold: read three
// times, the second and third time from the caches.
template <typename E>
__global__ __launch_bounds__(1024) void norm_long_kernel(const NormDesc D)
{
    constexpr int N = 16 / sizeof(E), LANES = 1024;
    __shared__ float lds[2][LANES / 64];
    const uint32_t t = blockIdx.x;
    const char *x = D.x + uint64_t(t) * D.row;
    float sum[1] = {0.f}, sq[1] = {0.f};
    for (int pass = 0; pass < 2; ++pass) {
        const float mean = sum[0] * D.inv_D;
        float s = 0.f;
        for (uint32_t a = threadIdx.x; a < D.vecs; a += LANES) {
            const uint32_t off = vec_offset<16>(a, D.row), seen = shared_front<E, 16>(a, off);
            float f[N];
            unpack<E, 16>(load_vec<16, false>(x + off), f);
#pragma unroll
            for (int i = 0; i < N; ++i)
                s += uint32_t(i) < seen ? 0.f : pass ? (f[i] - mean) * (f[i] - mean) : f[i];
        }
        if (pass) {
            sq[0] = s;
            team_sum<LANES, 1>(sq, lds[1]);
        } else {
            sum[0] = s;
            team_sum<LANES, 1>(sum, lds[0]);
        }
    }
    const float mean = sum[0] * D.inv_D, rstd = 1.f / sqrtf(sq[0] * D.inv_D + D.eps);
    for (uint32_t a = threadIdx.x; a < D.vecs; a += LANES) {
        const uint32_t off = vec_offset<16>(a, D.row);
        float w[N], b[N];
        load_weights<E, 16>(D, off, w, b);
        norm_vector<E, 16>(load_vec<16, false>(x + off), mean, rstd, w, b, D.y + uint64_t(t) * D.row + off);
    }
    if (threadIdx.x == 0) {
        if (D.mean)
            D.mean[t] = mean;
        if (D.rstd)
            D.rstd[t] = rstd;
    }
}

// --------------------------------------------------------------- gradient --

struct NormGradDesc {
    const char *dy, *x;
    const void *weight;
    const float *mean, *rstd;
    char *dx;
    float *partial;                 // [groups][2][width], the weight's and the bias's
    uint64_t rows;
    uint32_t groups, row, vecs, D, width;
    float inv_D;
    basp_dtype weight_dtype;
};

// Columns of a work-group's partial sums from vectors of a row: those of a
// vector that the one before holds too are left to it.
template <typename E, int VW, int N>
__device__ inline void store_columns(float *to, uint32_t a, uint32_t off, const float (&f)[N])
{
    const uint32_t seen = shared_front<E, VW>(a, off);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (uint32_t(i) >= seen)
            to[off / sizeof(E) + i] = f[i];
}

// LANES lanes take a row, R vectors each; a work-group's teams take rows in
// turn and keep the sums over them in registers; the next rows are on their way
// while some are summed.  32768 rows of 2048 in bf16: 72 us, 5.6 TB/s (89 us with
// 64 lanes a row, two work-groups of 256 a compute unit in both); 4099 rows of 777
// in fp32, which end inside vectors: 12 us, half of it before the first rows are
// there and after the last.
template <typename E, int VW, int LANES, int R, int THREADS>
__global__ __launch_bounds__(THREADS, 2) void norm_grad_kernel(const NormGradDesc D)
{
    constexpr int N = VW / sizeof(E), TEAMS = THREADS / LANES, COLUMNS = LANES * N;
    constexpr bool AHEAD = R <= 2;              // more would not fit in registers
    __shared__ float lds[2][LANES > 64 ? THREADS / 64 * 2 : 1];
    __shared__ float joined[TEAMS > 1 ? TEAMS : 1][TEAMS > 1 ? COLUMNS * 2 : 1];
    const uint32_t lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
    uint32_t off[R], seen[R];
    float w[R][N], dw[R][N], db[R][N];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint32_t a = lane + r * LANES;
        off[r] = vec_offset<VW>(a, D.row);
        seen[r] = a < D.vecs ? shared_front<E, VW>(a, off[r]) : N;
#pragma unroll
        for (int i = 0; i < N; ++i)
            w[r][i] = dw[r][i] = db[r][i] = 0.f;
        if (a < D.vecs)
            load_any<N>(D.weight, off[r] / sizeof(E), D.weight_dtype, w[r]);
    }
    typename MemVec<VW>::type xv[R] = {}, gv[R] = {}, next_x[R] = {}, next_g[R] = {};
    float next_mean = 0.f, next_rstd = 0.f;
    const auto fetch = [&](uint64_t t) {
        if (t >= D.rows)
            return;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (lane + r * LANES < D.vecs) {
                next_g[r] = load_vec<VW, true>(D.dy + t * D.row + off[r]);
                next_x[r] = load_vec<VW, true>(D.x + t * D.row + off[r]);
            }
        next_mean = D.mean[t];
        next_rstd = D.rstd[t];
    };
    const uint64_t step = uint64_t(D.groups) * TEAMS;
    if constexpr (AHEAD)
        fetch(uint64_t(blockIdx.x) * TEAMS + team);
    int turn = 0;
    for (uint64_t first = uint64_t(blockIdx.x) * TEAMS; first < D.rows; first += step, turn ^= 1) {
        const uint64_t t = first + team;
        const bool live = t < D.rows;
        const uint64_t at = t * D.row;
        if constexpr (!AHEAD)
            fetch(t);
        const float mean = next_mean, rstd = live ? next_rstd : 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            xv[r] = next_x[r];
            gv[r] = next_g[r];
            if (!live)
                gv[r] = {};
        }
        if constexpr (AHEAD)
            fetch(t + step);
        float sums[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float x[N], g[N];
            unpack<E, VW>(xv[r], x);
            unpack<E, VW>(gv[r], g);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float xhat = (x[i] - mean) * rstd, gw = g[i] * w[r][i];
                dw[r][i] = fmaf(g[i], xhat, dw[r][i]);
                db[r][i] += g[i];
                sums[0] += uint32_t(i) < seen[r] ? 0.f : gw;
                sums[1] += uint32_t(i) < seen[r] ? 0.f : gw * xhat;
            }
        }
        team_sum<LANES, 2>(sums, lds[turn]);
        const float c1 = sums[0] * D.inv_D, c2 = sums[1] * D.inv_D;
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (live && lane + r * LANES < D.vecs) {
                float x[N], g[N];
                unpack<E, VW>(xv[r], x);
                unpack<E, VW>(gv[r], g);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    x[i] = rstd * (g[i] * w[r][i] - c1 - (x[i] - mean) * rstd * c2);
                store_vec<VW>(D.dx + at + off[r], pack<E, VW>(x));
            }
    }
    float *const mine = D.partial + uint64_t(blockIdx.x) * 2 * D.width;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if constexpr (TEAMS == 1) {
            if (lane + r * LANES < D.vecs) {
                store_columns<E, VW>(mine, lane + r * LANES, off[r], dw[r]);
                store_columns<E, VW>(mine + D.width, lane + r * LANES, off[r], db[r]);
            }
        } else {                    // the teams' sums, added in their order
            lds_barrier();
#pragma unroll
            for (int i = 0; i < N; ++i) {
                joined[team][i * LANES + lane] = dw[r][i];
                joined[team][COLUMNS + i * LANES + lane] = db[r][i];
            }
            lds_barrier();
            for (uint32_t c = threadIdx.x; c < COLUMNS * 2; c += THREADS) {
                float sum = joined[0][c];
                for (int j = 1; j < TEAMS; ++j)
                    sum += joined[j][c];
                const uint32_t a = c % LANES + r * LANES, i = c / LANES % N, at = vec_offset<VW>(a, D.row);
                if (a < D.vecs && i >= shared_front<E, VW>(a, at))
                    mine[(c >= COLUMNS ? D.width : 0) + at / sizeof(E) + i] = sum;
            }
        }
    }
}

// Long rows: the gradient of x, a row a work-group, read twice.
template <typename E>
__global__ __launch_bounds__(1024) void norm_grad_long_kernel(const NormGradDesc D)
{
    constexpr int N = 16 / sizeof(E), LANES = 1024;
    __shared__ float lds[LANES / 64 * 2];
    const uint64_t t = blockIdx.x;
    const float mean = D.mean[t], rstd = D.rstd[t];
    float sums[2] = {0.f, 0.f};
    for (int pass = 0; pass < 2; ++pass) {
        for (uint32_t a = threadIdx.x; a < D.vecs; a += LANES) {
            const uint32_t off = vec_offset<16>(a, D.row), seen = shared_front<E, 16>(a, off);
            float x[N], g[N], w[N];
            unpack<E, 16>(load_vec<16, false>(D.x + t * D.row + off), x);
            unpack<E, 16>(load_vec<16, false>(D.dy + t * D.row + off), g);
            load_any<N>(D.weight, off / sizeof(E), D.weight_dtype, w);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float xhat = (x[i] - mean) * rstd, gw = g[i] * w[i];
                if (pass) {
                    x[i] = rstd * (gw - sums[0] * D.inv_D - xhat * (sums[1] * D.inv_D));
                } else {
                    sums[0] += uint32_t(i) < seen ? 0.f : gw;
                    sums[1] += uint32_t(i) < seen ? 0.f : gw * xhat;
                }
            }
            if (pass)
                store_vec<16>(D.dx + t * D.row + off, pack<E, 16>(x));
        }
        if (!pass)
            team_sum<LANES, 2>(sums, lds);
    }
}

// Long rows: the partial sums, a vector of columns a lane and every groups-th row.
template <typename E>
__global__ __launch_bounds__(kThreads) void norm_columns_kernel(const NormGradDesc D)
{
    constexpr int N = 16 / sizeof(E);
    const uint32_t a = blockIdx.x * kThreads + threadIdx.x;
    if (a >= D.vecs)
        return;
    const uint32_t off = vec_offset<16>(a, D.row);
    float dw[N] = {}, db[N] = {};
    for (uint64_t t = blockIdx.y; t < D.rows; t += D.groups) {
        const float mean = D.mean[t], rstd = D.rstd[t];
        float x[N], g[N];
        unpack<E, 16>(load_vec<16, false>(D.x + t * D.row + off), x);
        unpack<E, 16>(load_vec<16, false>(D.dy + t * D.row + off), g);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            dw[i] = fmaf(g[i], (x[i] - mean) * rstd, dw[i]);
            db[i] += g[i];
        }
    }
    float *const mine = D.partial + uint64_t(blockIdx.y) * 2 * D.width;
    store_columns<E, 16>(mine, a, off, dw);
    store_columns<E, 16>(mine + D.width, a, off, db);
}

struct NormJoinDesc {
    const float *partial;
    void *dweight, *dbias;
    uint32_t groups, D, width;
    basp_dtype weight_dtype;
};

// Sums of the work-groups' partial sums: 16 lanes side by side take four
// columns each, and 16 of them every sixteenth work-group.  blockIdx.y: the
// weight's or the bias's.  4 to 5 us for 512 x 2048, a launch and its latency.
__global__ __launch_bounds__(kThreads) void norm_join_kernel(const NormJoinDesc D)
{
    typedef float f4 __attribute__((ext_vector_type(4)));
    __shared__ f4 part[16][16];
    const uint32_t c = threadIdx.x & 15, s = threadIdx.x >> 4, col = (blockIdx.x * 16 + c) * 4;
    f4 sum = {0.f, 0.f, 0.f, 0.f};
    if (col < D.width)
#pragma unroll 8
        for (uint32_t g = s; g < D.groups; g += 16)
            sum += *reinterpret_cast<const f4 *>(D.partial + (uint64_t(g) * 2 + blockIdx.y) * D.width + col);
    part[s][c] = sum;
    lds_barrier();
    void *const to = blockIdx.y ? D.dbias : D.dweight;
    if (s == 0 && to) {
        for (int j = 1; j < 16; ++j)
            sum += part[j][c];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < D.D)
                store_number(to, col + i, D.weight_dtype, sum[i]);
    }
}

// --------------------------------------------------------------- launches --

// fn for a row of `vecs` vectors: f(lanes of a row, function).  Lanes and
// vectors a lane so that a row is in registers at once.
struct NormShape {
    const void *fn;
    int lanes;                      // or threads, of a gradient
    int groups;                     // that take rows in turn: as many as the device holds at once
};

template <typename E, int VW>
NormShape norm_shape(int64_t vecs)
{
    const auto of = [](auto fn, int lanes, int groups) { return NormShape{reinterpret_cast<const void *>(fn), lanes, groups}; };
    if (vecs <= 16)
        return of(norm_kernel<E, VW, 16, 1>, 16, 2048);
    if constexpr (VW == 16) {
        if (vecs <= 64)
            return of(norm_kernel<E, VW, 64, 1>, 64, 2048);
        if (vecs <= 128)
            return of(norm_kernel<E, VW, 64, 2>, 64, 1024);
        if (vecs <= 256)
            return of(norm_kernel<E, VW, 256, 1>, 256, 2048);
        if (vecs <= 512)
            return of(norm_kernel<E, VW, 256, 2>, 256, 1024);
        if (vecs <= 1024)
            return of(norm_kernel<E, VW, 256, 4>, 256, 512);
        if (vecs <= 2048)                   // 8192 rows of 16384 in bf16: 91 us, 226 us as long rows
            return of(norm_kernel<E, VW, 512, 4>, 512, 256);
        if (vecs <= 4096)
            return of(norm_kernel<E, VW, 1024, 4>, 1024, 256);
    }
    return of(norm_long_kernel<E>, 1024, 0);
}

template <typename E, int VW>
NormShape norm_grad_shape(int64_t vecs)
{
    const auto of = [](auto fn, int threads) { return NormShape{reinterpret_cast<const void *>(fn), threads, 0}; };
    if (vecs <= 16)
        return of(norm_grad_kernel<E, VW, 16, 1, 256>, 256);
    if constexpr (VW == 16) {
        if (vecs <= 64)
            return of(norm_grad_kernel<E, VW, 64, 1, 256>, 256);
        if (vecs <= 128)
            return of(norm_grad_kernel<E, VW, 64, 2, 256>, 256);
        if (vecs <= 256)
            return of(norm_grad_kernel<E, VW, 128, 2, 256>, 256);
        if (vecs <= 512)
            return of(norm_grad_kernel<E, VW, 256, 2, 256>, 256);
        if (vecs <= 1024)
            return of(norm_grad_kernel<E, VW, 512, 2, 512>, 512);
        // 8192 rows of 12288 in bf16: 230 us although it spills, 260 us as 1024 x 2,
        // which spills more, 302 us as long rows; of 8192 in fp32: 150 us
        if (vecs <= kNormGradVecs)
            return of(norm_grad_kernel<E, VW, sizeof(E) == 2 ? 512 : 1024, sizeof(E) == 2 ? 4 : 2, sizeof(E) == 2 ? 512 : 1024>,
                      sizeof(E) == 2 ? 512 : 1024);
    }
    return of(norm_grad_long_kernel<E>, 1024);
}

template <typename E>
const void *columns_fn()
{
    return reinterpret_cast<const void *>(norm_columns_kernel<E>);
}

basp_status launch_norm(const basp_norm_plan &p, const void *x, const void *weight, const void *bias, float eps, void *y,
                        float *mean, float *rstd, void *stream)
{
    const int64_t row = p.D * p.es;
    const NormShape s = BASP_BY_ROW(norm_shape, p.dtype, p.vw, p.vecs);
    const bool in_turn = s.groups > 0;                  // or a row a work-group
    const int64_t teams = std::max(kThreads / s.lanes, 1), step = in_turn ? p.T : kLaunchGroups / 4;
    basp_status st = BASP_OK;
    for (int64_t t0 = 0; t0 < p.T && st == BASP_OK; t0 += step) {
        const int64_t n = std::min(step, p.T - t0), groups = (n + teams - 1) / teams;
        const NormDesc D = {static_cast<const char *>(x) + t0 * row, weight, bias, static_cast<char *>(y) + t0 * row,
                            mean ? mean + t0 : nullptr, rstd ? rstd + t0 : nullptr, uint32_t(n), uint32_t(row),
                            uint32_t(p.vecs), uint32_t(p.D), eps, 1.f / float(p.D), p.weight_dtype};
        st = launch_kernel(s.fn, dim3(uint32_t(in_turn ? std::min<int64_t>(groups, s.groups) : groups)),
                           std::max(kThreads, s.lanes), D, stream, t0 == 0, t0 + n == p.T);
    }
    return st;
}

basp_status launch_norm_grad(const basp_norm_plan &p, const void *dy, const void *x, const void *weight, const float *mean,
                             const float *rstd, void *dx, void *dweight, void *dbias, void *ws, void *stream)
{
    const int64_t row = p.D * p.es;
    const NormShape s = BASP_BY_ROW(norm_grad_shape, p.dtype, p.vw, p.vecs);
    NormGradDesc D = {static_cast<const char *>(dy), static_cast<const char *>(x), weight, mean, rstd, static_cast<char *>(dx),
                      static_cast<float *>(ws), uint64_t(p.T), uint32_t(p.grad_groups), uint32_t(row), uint32_t(p.vecs),
                      uint32_t(p.D), uint32_t(p.width), 1.f / float(p.D), p.weight_dtype};
    basp_status st = BASP_OK;
    if (p.T && (p.vecs <= kNormGradVecs || p.vw < 16)) {
        st = launch_kernel(s.fn, dim3(D.groups), s.lanes, D, stream, true, false);
    } else if (p.T) {
        const int64_t step = kLaunchGroups / 4;
        for (int64_t t0 = 0; t0 < p.T && st == BASP_OK; t0 += step) {
            NormGradDesc part = D;
            part.dy += t0 * row;
            part.x += t0 * row;
            part.dx += t0 * row;
            part.mean += t0;
            part.rstd += t0;
            st = launch_kernel(s.fn, dim3(uint32_t(std::min(step, p.T - t0))), s.lanes, part, stream, t0 == 0, false);
        }
        const void *fn = p.dtype == BASP_FP32 ? columns_fn<float>() : p.dtype == BASP_BF16 ? columns_fn<__bf16>() : columns_fn<_Float16>();
        if (st == BASP_OK)
            st = launch_kernel(fn, dim3(uint32_t((p.vecs + kThreads - 1) / kThreads), D.groups), kThreads, D, stream, false, false);
    }
    const NormJoinDesc J = {D.partial, dweight, dbias, D.groups, D.D, D.width, p.weight_dtype};
    if (st == BASP_OK)
        st = launch_kernel(reinterpret_cast<const void *>(norm_join_kernel), dim3(uint32_t((p.width + 63) / 64), dbias ? 2 : 1),
                           kThreads, J, stream, p.T == 0, true);
    return st;
}

}  // namespace
}  // namespace basp

using basp::CallBuf;

extern "C" basp_status basp_layer_norm(const basp_norm_plan *p, const void *x, const void *weight, const void *bias,
                                       float eps, void *y, float *mean, float *rstd, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p || !(eps >= 0.f) || std::isinf(eps))
            return BASP_ERR_INVALID;
        const int64_t rows = p->T * p->D * p->es, cols = p->D * p->ws_es, stats = p->T * 4;
        const CallBuf in[] = {{x, rows, p->es}, {weight, cols, p->ws_es}, {bias, bias ? cols : 0, p->ws_es}};
        const CallBuf out[] = {{y, rows, p->es}, {mean, mean ? stats : 0, 4}, {rstd, rstd ? stats : 0, 4}};
        const basp_status s = basp::check_call(in, 3, out, 3);
        return s != BASP_OK ? s : basp::launch_norm(*p, x, weight, bias, eps, y, mean, rstd, stream);
    });
}

extern "C" basp_status basp_layer_norm_grad(const basp_norm_plan *p, const void *dy, const void *x, const void *weight,
                                            const float *mean, const float *rstd, void *dx, void *dweight, void *dbias,
                                            void *ws, void *stream)
{
    return basp::timed_call([&]() -> basp_status {
        if (!p)
            return BASP_ERR_INVALID;
        const int64_t rows = p->T * p->D * p->es, cols = p->D * p->ws_es, stats = p->T * 4;
        const CallBuf in[] = {{dy, rows, p->es}, {x, rows, p->es}, {weight, cols, p->ws_es}, {mean, stats, 4}, {rstd, stats, 4}};
        const CallBuf out[] = {{dx, rows, p->es}, {dweight, cols, p->ws_es}, {dbias, dbias ? cols : 0, p->ws_es},
                               {ws, p->workspace_bytes, 16}};
        const basp_status s = basp::check_call(in, 5, out, 4);
        return s != BASP_OK ? s : basp::launch_norm_grad(*p, dy, x, weight, mean, rstd, dx, dweight, dbias, ws, stream);
    });
}
