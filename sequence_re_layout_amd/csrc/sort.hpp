// sort.hpp -- a stable sort of items by a small integer (an expert, or one
// digit of a vocabulary id), as one work-group sees its share of it.
//
// Item i of bin e goes to   start[e] + #{items j < i of bin e},   start being
// the running sum of the bins' counts, each rounded up to a multiple of
// `align`.  A work-group takes consecutive items and each of its waves a
// consecutive part of those, so the rank of an item is the sum of four
// counts: the bin's start, the bin's items in earlier work-groups, in earlier
// waves of this one, and in the wave's own earlier items.  The last is kept
// in LDS, one counter per wave and bin, and within 64 items comes from a
// match: one ballot per bit of the bin leaves each lane the mask of the lanes
// that hold the same bin.  No atomic decides an order, so the result is the
// stable one on every run.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "barrier.hpp"
#include "index_plan.hpp"

namespace basp {

// LDS of one work-group: counters [waves][bins], the bins' totals, starts
// (bins + 1) and a scratch word per wave.
struct SortLds {
    int *count, *total, *start, *scan;
};

inline size_t sort_lds_bytes(int waves, int bins) { return 4 * (size_t(waves) * bins + bins + bins + 1 + waves); }

__device__ inline SortLds sort_lds(int *mem, int waves, int bins)
{
    SortLds l;
    l.count = mem;
    l.total = l.count + waves * bins;
    l.start = l.total + bins;
    l.scan = l.start + bins + 1;
    return l;
}

__device__ inline int wave_inclusive_sum(int v, int lane)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        v += lane >= d ? o : 0;
    }
    return v;
}

// The lanes of the wave that hold the same bin (bins of `bits` bits); only
// lanes with bin >= 0 count.
__device__ inline uint64_t same_bin(int bin, int bits)
{
    uint64_t m = __ballot(bin >= 0);
    for (int b = 0; b < bits; ++b) {
        const int bit = (bin >> b) & 1;
        const uint64_t v = __ballot(bit);
        const uint32_t flip = bit - 1;      // all ones where the bit is clear
        m &= v ^ (uint64_t{flip} << 32 | flip);
    }
    return m;
}

__device__ inline int lds_get(int *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT); }
__device__ inline void lds_put(int *p, int v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
}

// The bins' totals over all work-groups and their counts in the groups before
// this one, into l.total and l.start.  A thread keeps to one bin (or one of
// every WAVES * 64), so that a bin's counts meet in few atomics.
template <int WAVES>
__device__ inline void sort_sum_groups(const SortLds &l, const int *hist, int bins, int groups, int group)
{
    constexpr int NT = WAVES * 64;
    int span = 1;                       // threads of one group's counts
    while (span < bins && span < NT)
        span <<= 1;
    const int rows = NT / span, g0 = threadIdx.x / span;
    constexpr int U = 16;               // counts in flight
    for (int e = threadIdx.x & (span - 1); e < bins; e += span) {
        int total = 0, before = 0;
        for (int g1 = g0; g1 < groups; g1 += U * rows) {
            int n[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int g = g1 + u * rows;
                n[u] = g < groups ? hist[int64_t{g} * bins + e] : 0;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                total += n[u];
                before += g1 + u * rows < group ? n[u] : 0;
            }
        }
        if (rows == 1) {
            l.total[e] = total;
            l.start[e] = before;
        } else if (total) {
            atomicAdd(&l.total[e], total);
            atomicAdd(&l.start[e], before);
        }
    }
}

// From the waves' counts (l.count), and with more than one group the totals
// and the counts before this group: the starts, an exclusive sum over the
// bins, a few consecutive ones a thread; and in l.count the place of each
// wave's next item of a bin.
template <int WAVES>
__device__ inline void sort_starts(const SortLds &l, int bins, int align, int groups)
{
    constexpr int NT = WAVES * 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int per = (bins + NT - 1) / NT, e0 = tid * per;
    const bool has = wave * 64 * per < bins;     // the wave has bins
    int sum = 0;
    if (has) {
        for (int j = 0; j < per && e0 + j < bins; ++j) {
            const int e = e0 + j;
            if (groups == 1) {
                int n = 0;
#pragma unroll
                for (int w = 0; w < WAVES; ++w)
                    n += l.count[w * bins + e];
                l.total[e] = n;
            }
            sum += padded_count(l.total[e], align);
        }
        const int upto = wave_inclusive_sum(sum, lane);
        if (lane == 63)
            l.scan[wave] = upto;
        sum = upto - sum;
    }
    lds_barrier();
    if (has) {
        int at = sum;
        for (int w = 0; w < wave; ++w)
            at += l.scan[w];
        for (int j = 0; j < per && e0 + j < bins; ++j) {
            const int e = e0 + j;
            int next = at + (groups == 1 ? 0 : l.start[e]);
            int n[WAVES];               // read before the first is written: one wait for all
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
                n[w] = l.count[w * bins + e];
            const int total = l.total[e];
            l.start[e] = at;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                l.count[w * bins + e] = next;
                next += n[w];
            }
            at += padded_count(total, align);
            if (e == bins - 1)
                l.start[bins] = at;
        }
    }
    lds_barrier();
}

__device__ inline int bits_of(int bins)
{
    int bits = 0;
    while ((bins - 1) >> bits)
        ++bits;
    return bits;
}

// One step of a wave: the rank of each lane's item among the wave's items of
// its bin so far, counted in `mine`.  Lanes without an item pass bin -1.
__device__ inline int wave_rank(int *mine, int bin, int bits, uint64_t below)
{
    const uint64_t same = same_bin(bin, bits);
    int first = 0;
    const int rank = __popcll(same & below);
    if (bin >= 0) {
        first = lds_get(&mine[bin]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (rank == 0)
            lds_put(&mine[bin], first + __popcll(same));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return first + rank;
}

// Places the items [begin, end) of work-group `group` of `groups`.
//   key(i)            what the item carries
//   bin(key)          its bin in [0, bins), or -1: not placed
//   hist              counts [groups][bins] of every work-group; not read
//                     where groups is 1
//   emit(i, key, at)  called once for every item; at is -1 if not placed
// Returns with l.total and l.start (bins + 1 entries) filled for all threads.
// All WAVES * 64 threads call it.  R > 0: there are at most WAVES * 64 * R
// items, and a wave reads its R * 64 once, ranks them as it counts them and
// keeps both in registers; R = 0: any number, read twice.
template <int WAVES, int R, typename Key, typename Bin, typename Emit>
__device__ inline void sort_place(const SortLds &l, int64_t begin, int64_t end, int bins, int align,
                                  const int *hist, int groups, int group, Key key, Bin bin, Emit emit)
{
    constexpr int NT = WAVES * 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint64_t below = (uint64_t{1} << lane) - 1;
    const int bits = bits_of(bins);
    int *const mine = l.count + wave * bins;
    const int64_t part = (end - begin + NT - 1) / NT * 64;
    const int64_t w0 = begin + wave * part, w1 = w0 + part < end ? w0 + part : end;
    if constexpr (R > 0) {
        decltype(key(int64_t{0})) k[R > 0 ? R : 1];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t i = w0 + r * 64 + lane;
            k[r] = i < w1 ? key(i) : 0;
        }
        for (int i = tid; i < WAVES * bins; i += NT)
            l.count[i] = 0;
        for (int i = tid; i < bins; i += NT)
            l.total[i] = l.start[i] = 0;
        lds_barrier();
        if (groups > 1)
            sort_sum_groups<WAVES>(l, hist, bins, groups, group);
        int rank[R > 0 ? R : 1];
#pragma unroll
        for (int r = 0; r < R; ++r)
            if (w0 + r * 64 < w1)        // the same for all lanes of a wave
                rank[r] = wave_rank(mine, w0 + r * 64 + lane < w1 ? bin(k[r]) : -1, bits, below);
        lds_barrier();
        sort_starts<WAVES>(l, bins, align, groups);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t i = w0 + r * 64 + lane;
            if (i < w1) {
                const int e = bin(k[r]);
                emit(i, k[r], e < 0 ? -1 : mine[e] + rank[r]);
            }
        }
    } else {
        for (int i = tid; i < WAVES * bins; i += NT)
            l.count[i] = 0;
        for (int i = tid; i < bins; i += NT)
            l.total[i] = l.start[i] = 0;
        lds_barrier();
        if (groups > 1)
            sort_sum_groups<WAVES>(l, hist, bins, groups, group);
        for (int64_t i = w0 + lane; i < w1; i += 64) {
            const int e = bin(key(i));
            if (e >= 0)
                atomicAdd(&mine[e], 1);
        }
        lds_barrier();
        sort_starts<WAVES>(l, bins, align, groups);
        for (int64_t i0 = w0; i0 < w1; i0 += 64) {   // the same for all lanes of a wave
            const int64_t i = i0 + lane;
            decltype(key(int64_t{0})) k = 0;
            int e = -1;
            if (i < w1) {
                k = key(i);
                e = bin(k);
            }
            const int at = wave_rank(mine, e, bits, below);
            if (i < w1)
                emit(i, k, e < 0 ? -1 : at);
        }
    }
}

// The counts of one work-group's items, for the sort of many groups.
// bin(i): the bin of item i, or -1.
template <int WAVES, typename Bin>
__device__ inline void sort_count(int *count, int64_t begin, int64_t end, int bins, int *hist, Bin bin)
{
    constexpr int NT = WAVES * 64, U = 4;
    for (int i = threadIdx.x; i < bins; i += NT)
        count[i] = 0;
    lds_barrier();
    for (int64_t i0 = begin + threadIdx.x; i0 < end; i0 += NT * U) {
        int e[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            e[u] = i0 + u * NT < end ? bin(i0 + u * NT) : -1;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (e[u] >= 0)
                atomicAdd(&count[e[u]], 1);
    }
    lds_barrier();
    for (int i = threadIdx.x; i < bins; i += NT)
        hist[i] = count[i];
}

}  // namespace basp
