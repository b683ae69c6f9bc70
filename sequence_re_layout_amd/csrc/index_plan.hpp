// index_plan.hpp -- the plans of the index-driven re-layouts and the index
// arithmetic their kernels share with the host.
#pragma once

#include <cstdint>

#ifndef BASP_HD
#define BASP_HD
#endif
#include "basp.h"
#include "fastdiv.hpp"

// T tokens, K choices each, E experts, rows of D channels (basp.h).
struct basp_expert_plan {
    int64_t T, D;
    int32_t K, E, align, id_bytes;
    basp_dtype dtype, weight_dtype;
    int32_t es, ws_es;              // element sizes of rows and weights
    int64_t slots, max_rows;
    int32_t sort_blocks;            // work-groups of a sort
    int64_t block_items;            // slots of one of them
    int64_t workspace_bytes;
};

// Where token t of the order [B][S] lies in the sequence-sharded layout
// (basp.h, "Memory layouts"): member j of group g holds the tokens
// [j*St, (j+1)*St) of its group's Bl sequences.
struct basp_seq_order {
    int32_t same;                   // the orders are the same
    uint32_t P, St, Bl, S;
    basp::FastDiv by_S, by_Bl, by_St;
};

struct basp_embed_plan {
    int64_t T, V, D, padding;
    int32_t id_bytes;
    basp_dtype dtype, grad_dtype;
    int32_t es, grad_es;
    basp_seq_order order;
    int32_t passes, digit_bits;     // of the sort by id
    int32_t sort_blocks;
    int64_t block_items;
    int64_t chunks;                 // groups of tokens that are summed in one go
    int64_t width;                  // channels of a partial sum, whole vectors
    // byte offsets in the workspace
    int64_t keys[2], tokens[2], hist, partials;
    int64_t workspace_bytes;
};

namespace basp {

constexpr int kSortWaves = 8;               // waves of a sort's work-group
constexpr int kSortBlock = 64 * kSortWaves;
constexpr int kMaxExperts = 1024;           // and digits of one pass of a sort
constexpr int kChunk = 32;                  // tokens summed in one go

BASP_HD inline uint32_t seq_row(const basp_seq_order &o, uint32_t t)
{
    if (o.same)
        return t;
    const uint32_t seq = fastdiv(t, o.by_S), at = t - seq * o.S;
    const uint32_t g = fastdiv(seq, o.by_Bl), j = fastdiv(at, o.by_St);
    return ((g * o.P + j) * o.Bl + (seq - g * o.Bl)) * o.St + (at - j * o.St);
}

// Rows are read and written in vectors of vw bytes, the widest power of two
// up to 16 that a row holds one of.  A row of `elems` elements takes
// ceil(elems / epv) vectors; the last one ends with the row and so overlaps
// the one before it where the row is no whole number of vectors.  Copies and
// sums write the same bits twice there.
inline int row_vector(int64_t D, int es)
{
    int vw = 16;
    while (vw > es && D * es < vw)
        vw /= 2;
    return vw;
}

// Buffers of a call: NULL, alignment and aliasing checks (basp.h,
// "Conventions common to every call").
struct CallBuf {
    const void *ptr;
    int64_t bytes;
    int align;
};
basp_status check_call(const CallBuf *in, int nin, const CallBuf *out, int nout);

}  // namespace basp
