// teams.hpp -- sums over the lanes that share a row: part of a wave, a wave, or
// a whole work-group.
#pragma once

#include <hip/hip_runtime.h>

#include "barrier.hpp"
#include "rowvec.hpp"

namespace basp {

// f of x and the x of the lanes D away (the mirrored lane for 4 and 8, where
// closer lanes hold the same already), without a trip through LDS.
template <int D, typename F>
__device__ inline float with_lane(float x, F f)
{
    const int w = __builtin_bit_cast(int, x);
    if constexpr (D >= 16) {
        uint32_t a, b;
        if constexpr (D == 16) {
            const auto r = __builtin_amdgcn_permlane16_swap(uint32_t(w), uint32_t(w), false, false);
            a = r[0], b = r[1];
        } else {
            const auto r = __builtin_amdgcn_permlane32_swap(uint32_t(w), uint32_t(w), false, false);
            a = r[0], b = r[1];
        }
        return f(__builtin_bit_cast(float, a), __builtin_bit_cast(float, b));
    } else {
        // quad_perm [1,0,3,2] and [2,3,0,1], row_half_mirror, row_mirror
        constexpr int WAY = D == 1 ? 0xb1 : D == 2 ? 0x4e : D == 4 ? 0x141 : 0x140;
        return f(x, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, w, WAY, 0xf, 0xf, true)));
    }
}

// Sums over the lanes of a wave that are multiples of LANES apart.
template <int LANES>
__device__ inline float sum_of_teams(float x)
{
    const auto add = [](float a, float b) { return a + b; };
    if constexpr (LANES <= 8) {
        // row_ror:8 and row_ror:4: around in 16 lanes
        x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x128, 0xf, 0xf, true));
        if constexpr (LANES <= 4)
            x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x124, 0xf, 0xf, true));
    }
    if constexpr (LANES <= 16)
        x = with_lane<16>(x, add);
    if constexpr (LANES <= 32)
        x = with_lane<32>(x, add);
    return x;
}

// x of the lanes of a team, or of a wave, put together by f; the same bits in all.
template <int LANES, typename F>
__device__ inline float team_fold(float x, F f)
{
    if constexpr (LANES > 1)
        x = with_lane<1>(x, f);
    if constexpr (LANES > 2)
        x = with_lane<2>(x, f);
    if constexpr (LANES > 4)
        x = with_lane<4>(x, f);
    if constexpr (LANES > 8)
        x = with_lane<8>(x, f);
    if constexpr (LANES > 16)
        x = with_lane<16>(x, f);
    if constexpr (LANES > 32)
        x = with_lane<32>(x, f);
    return x;
}

// Sums of M numbers over a team of LANES lanes, the same bits in every lane.
// `lds` holds M numbers a wave where a team has several; calls that follow each
// other need the two halves of a pair in turn.
template <int LANES, int M>
__device__ inline void team_sum(float (&x)[M], float *lds)
{
#pragma unroll
    for (int m = 0; m < M; ++m)
        x[m] = team_fold<LANES>(x[m], [](float a, float b) { return a + b; });
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
