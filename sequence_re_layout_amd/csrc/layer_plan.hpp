// layer_plan.hpp -- the plans of the layer norm (and the sizes that the balance
// loss of an expert plan needs), in plain C++.
#pragma once

#include <cstdint>

#include "basp.h"
#include "index_plan.hpp"

struct basp_norm_plan {
    int64_t T, D;
    basp_dtype dtype, weight_dtype;
    int32_t es, ws_es;
    int32_t vw;                     // bytes of a vector of a row
    int64_t vecs;                   // vectors of a row, the last may overlap the one before
    int32_t grad_groups;            // partial sums of the weight's gradient
    int64_t width;                  // numbers of one of them
    int64_t workspace_bytes;
};

namespace basp {

inline int float_bytes(basp_dtype t)
{
    return t == BASP_BF16 || t == BASP_FP16 ? 2 : t == BASP_FP32 ? 4 : 0;
}

// Work-groups whose rows' shares of the weight's gradient are summed apart: two
// a compute unit (32768 x 2048 in bf16: see norm.hip).
constexpr int kNormGradGroups = 512;
// Vectors that the one-pass gradient holds in registers; longer rows are read
// again by columns.
constexpr int64_t kNormGradVecs = 2048;

// The balance loss: tokens are summed in up to 256 work-groups of
// kBalanceThreads, one partial sum and one count of every expert each, and one
// more work-group joins them, which reads about 130 GB/s: at most 2^17 of each.
constexpr int kBalanceThreads = 1024;

inline int balance_groups(const basp_expert_plan &p)
{
    const int64_t wanted = (p.T + 15) / 16, most = p.E <= 512 ? 256 : (int64_t{1} << 17) / p.E;
    return int(wanted < 1 ? 1 : wanted > most ? most : wanted);
}

}  // namespace basp
