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
    int32_t sort_blocks;            // work-groups of a pass; 0: sorted by counting alone
    int64_t block_items;
    int32_t lanes_log2;             // lanes of a team: one vector of channels each
    int32_t chunk;                  // sorted tokens that a team sums
    int64_t blocks;                 // of tokens, each with two partial sums
    int32_t col_groups;             // work-groups along the channels
    int64_t sum_groups;             // and of all
    int64_t width;                  // channels of a partial sum, whole vectors
    // byte offsets in the workspace
    int64_t keys[2], tokens[2], tags, hist, partials;
    int64_t workspace_bytes;
};

namespace basp {

constexpr int kSortWaves = 8;               // waves of a sort's work-group
constexpr int kSortBlock = 64 * kSortWaves;
constexpr int kSortSteps = 2;               // items of a lane that it keeps in registers: 2 or 8
constexpr int kSortItems = kSortBlock * kSortSteps;
constexpr int kMaxExperts = 1024;
constexpr int kDigitBits = 10;              // of one pass of a sort by id
// Tokens that are sorted by counting alone: with (id, token) pairs of 32 bits,
// and of 64, which fill 56 of the 64 KiB of LDS that a launch gets by default.
// Whole gradients by counting and by digits, us:
//   8191 x 128 (two digits)     4096 tokens 17.5 / 29.7, 8192 22.2 / 30.1, 11264
//                               29.5 / 30.5, 13500 37.8 / 30.6
//   2097152 x 8 (three)         4096 29.8 / 49.6, 7168 34.8 / 50.7
//   1000 x 128 (one)            4096 16.9 / 22.9, 8192 22.1 / 24.3, 11264 29.8 / 25.2
//   131072 x 2048 (two, beside  4096 96.5 / 97.7, 6000 101.2 / 98.5, 11264
//   512 MiB of zeros)           113.7 / 103.1
// The limit is that of the first kind: with one digit, or zeros that take as
// long as the digits, digits are faster from about 9000 and 5000 tokens on.
constexpr int kRankNarrow = 11264, kRankWide = 7168;

// Pairs id * T + token, ids up to V, in 32 bits.
inline bool fits_narrow(int64_t T, int64_t V) { return (V + 1) * T < int64_t{0xffffffff}; }
constexpr int kSumThreads = 256;
constexpr int kMerge = 8;                   // teams that join their sums in LDS, at most

// Teams of 2^lanes_log2 lanes.
inline int merged_teams(int lanes_log2)
{
    return (kSumThreads >> lanes_log2) < kMerge ? kSumThreads >> lanes_log2 : kMerge;
}

BASP_HD inline uint32_t seq_row(const basp_seq_order &o, uint32_t t)
{
    if (o.same)
        return t;
    const uint32_t seq = fastdiv(t, o.by_S), at = t - seq * o.S;
    const uint32_t g = fastdiv(seq, o.by_Bl), j = fastdiv(at, o.by_St);
    return ((g * o.P + j) * o.Bl + (seq - g * o.Bl)) * o.St + (at - j * o.St);
}

// n rounded up to a multiple of `to`, as a plan's slots and align are.  The sum
// passes 2^31 where one expert has nearly 2^31 slots, and always fits 32 bits
// without a sign; the result is at most max_rows.
BASP_HD inline int padded_count(int n, int to)
{
    return to == 1 ? n : int((uint32_t(n) + uint32_t(to) - 1) / uint32_t(to) * uint32_t(to));
}

// Bytes of a number of a floating type, 0 for any other.
inline int float_bytes(basp_dtype t)
{
    return t == BASP_BF16 || t == BASP_FP16 ? 2 : t == BASP_FP32 ? 4 : 0;
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

// Writing zeros into some rows of a buffer.  The buffer is cut into pieces of
// up to 4 KiB: several short rows, one row, or a part of a long one.  Four
// waves write a piece (or one wave a piece of short rows); neighbouring pieces
// belong to neighbouring work-groups, and a work-group's own `per` pieces lie
// `stride` pieces apart.  Measured on 512 MiB: 6.4-6.8 TB/s in this order,
// against 5.0-5.8 TB/s where a work-group writes 16 KiB or more in a row, and
// 4.1-4.7 TB/s from a grid that loops.
struct ZeroPieces {
    uint32_t row, rows, parts;      // bytes of a row; rows of a piece, or pieces of a row
    uint32_t begin, end;            // rows of the buffer
    uint32_t per, stride, groups;   // pieces of a work-group and how far apart; work-groups
    uint64_t pieces;
};

constexpr uint32_t kPiece = 4096;

inline ZeroPieces zero_pieces(int64_t begin, int64_t end, int64_t row, int waves)
{
    ZeroPieces z = {};
    const uint64_t n = uint64_t(end - begin);
    z.row = uint32_t(row);
    z.rows = row * 2 <= kPiece ? uint32_t(kPiece / row > 64 ? 64 : kPiece / row) : 1;
    z.parts = uint32_t((row + kPiece - 1) / kPiece);
    z.begin = uint32_t(begin);
    z.end = uint32_t(end);
    z.pieces = (n + z.rows - 1) / z.rows * z.parts;
    // one piece a wave, or four waves, while that does not fill the device
    z.per = z.rows > 1 ? uint32_t(z.pieces >= 4096 ? 8 : waves) : uint32_t(z.pieces >= 4096 ? waves / 2 : waves / 4);
    const uint64_t share = (z.pieces + z.per - 1) / z.per;
    z.stride = uint32_t(share > 256 ? 256 : share);
    const uint64_t sweeps = z.stride ? (share + z.stride - 1) / z.stride : 0;
    z.groups = z.stride * uint32_t(sweeps > 4096 ? 4096 : sweeps);
    return z;
}

// Piece number i of a work-group in its sweep s.
BASP_HD inline uint64_t zero_piece(const ZeroPieces &z, uint64_t s, uint32_t group, uint32_t i)
{
    return (s * z.per + i) * z.stride + group % z.stride;
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
