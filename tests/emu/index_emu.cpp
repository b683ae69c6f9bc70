// The host arithmetic of the index-driven re-layouts for tests without a GPU:
// the place of a token in the sequence-sharded layout, and which rows the
// work-groups of a launch look at when they write zeros.
#include <cstdint>
#include <cstring>

#include "index_plan.hpp"

using namespace basp;

extern "C" void emu_seq_rows(const basp_embed_plan *p, int64_t *out)
{
    for (int64_t t = 0; t < p->T; ++t)
        out[t] = seq_row(p->order, uint32_t(t));
}

// Counts, for every byte of rows [begin, end), how often write_zeros covers it
// with `waves` waves a work-group; seen has (end - begin) * row entries.
extern "C" int64_t emu_zero_cover(int64_t begin, int64_t end, int64_t row, int waves, uint8_t *seen)
{
    const ZeroPieces z = zero_pieces(begin, end, row, waves);
    int64_t bad = 0;
    for (uint32_t g = 0; g < z.groups; ++g)
        for (uint64_t s = g / z.stride; s * z.stride * z.per < z.pieces; s += z.groups / z.stride)
            for (uint32_t i = 0; i < z.per; ++i) {
                const uint64_t piece = zero_piece(z, s, g, i);
                if (piece >= z.pieces)
                    continue;
                int64_t r0, r1, b0 = 0, b1 = row;
                if (z.rows > 1) {
                    r0 = z.begin + int64_t(piece) * z.rows;
                    r1 = r0 + z.rows < z.end ? r0 + z.rows : z.end;
                } else {
                    r0 = z.begin + int64_t(piece / z.parts);
                    r1 = r0 + 1;
                    b0 = int64_t(piece % z.parts) * kPiece;
                    b1 = b0 + kPiece < row ? b0 + kPiece : row;
                }
                for (int64_t r = r0; r < r1; ++r)
                    for (int64_t b = b0; b < b1; ++b) {
                        if (r < begin || r >= end)
                            ++bad;
                        else
                            ++seen[(r - begin) * row + b];
                    }
            }
    return bad;
}
