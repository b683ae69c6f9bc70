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

// Work-groups whose rows' shares of the weight's gradient are summed apart: two
// a compute unit.
constexpr int kNormGradGroups = 512;
// Vectors of 16 bytes that the one-pass gradient holds in registers; longer rows
// are read again by columns.
constexpr int64_t kNormGradVecs = 2048;

// The balance loss.  A team of lanes takes a token's scores, up to four vectors a
// lane: sums over few lanes cost least, and with three or four vectors few lanes
// are idle.
constexpr int kBalanceThreads = 1024;

struct LogitRow {
    int vw;                         // bytes of a vector
    int64_t row, vecs;              // bytes and vectors of a token
    int lanes, regs;                // lanes of a team and vectors of a lane
};

inline LogitRow logit_row(const basp_expert_plan &p)
{
    LogitRow r;
    r.vw = row_vector(p.E, p.ws_es);
    r.row = int64_t{p.E} * p.ws_es;
    r.vecs = (r.row + r.vw - 1) / r.vw;
    r.lanes = r.vecs <= 4 ? 4 : r.vecs <= 32 ? 8 : r.vecs <= 64 ? 16 : r.vecs <= 128 ? 32 : 64;
    r.regs = int((r.vecs + r.lanes - 1) / r.lanes);
    return r;
}

// Tokens are summed in up to kBalanceGroups work-groups of kBalanceThreads, one
// partial sum and one count of every expert each; a second launch joins them.
// What one work-group does in a few steps is not worth that launch.
constexpr int kBalanceGroups = 256;

inline int balance_groups(const basp_expert_plan &p)
{
    const int64_t teams = kBalanceThreads / logit_row(p).lanes, wanted = p.T <= 4 * teams ? 1 : (p.T + teams - 1) / teams;
    return int(wanted > kBalanceGroups ? kBalanceGroups : wanted);
}

// Experts of a work-group that joins partial results; such work-groups.
constexpr int kJoinColumns = 32;
inline int balance_joins(const basp_expert_plan &p) { return p.E / kJoinColumns + 1; }

// Numbers of a partial result: a sum of every expert and a count, or the counts
// and the number of live tokens, in whole groups of four.
inline int64_t balance_stride(const basp_expert_plan &p) { return (int64_t{p.E} + 1 + 3) / 4 * 4; }

}  // namespace basp
