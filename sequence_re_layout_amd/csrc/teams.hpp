// teams.hpp -- sums over the lanes that share a row: part of a wave, a wave, or
// a whole work-group.
#pragma once

#include <hip/hip_runtime.h>

#include "barrier.hpp"
#include "rowvec.hpp"

namespace basp {

// Sums of M numbers over a team of LANES lanes, the same bits in every lane.
// `lds` holds M numbers a wave where a team has several; calls that follow each
// other need the two halves of a pair in turn.
template <int LANES, int M>
__device__ inline void team_sum(float (&x)[M], float *lds)
{
#pragma unroll
    for (int d = 1; d < (LANES < 64 ? LANES : 64); d <<= 1)
#pragma unroll
        for (int m = 0; m < M; ++m)
            x[m] += __shfl_xor(x[m], d);
    if constexpr (LANES > 64) {
        constexpr int WAVES = LANES / 64;
        const float *const team = lds + threadIdx.x / LANES * WAVES * M;
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int m = 0; m < M; ++m)
                lds[(threadIdx.x >> 6) * M + m] = x[m];
        lds_barrier();
#pragma unroll
        for (int m = 0; m < M; ++m) {
            float s = team[m];
#pragma unroll
            for (int w = 1; w < WAVES; ++w)
                s += team[w * M + m];
            x[m] = s;
        }
    }
}

template <int LANES>
__device__ inline float team_max(float x)
{
    static_assert(LANES <= 64, "a team of one wave");
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1)
        x = fmaxf(x, __shfl_xor(x, d));
    return x;
}

// N numbers from index i on, of a type known at run time, in fp32.
template <int N>
__device__ inline void load_any(const void *p, int64_t i, basp_dtype t, float (&f)[N])
{
    if (t == BASP_FP32)
        load_values<float, N>(static_cast<const char *>(p) + i * 4, f);
    else if (t == BASP_BF16)
        load_values<__bf16, N>(static_cast<const char *>(p) + i * 2, f);
    else
        load_values<_Float16, N>(static_cast<const char *>(p) + i * 2, f);
}

}  // namespace basp
