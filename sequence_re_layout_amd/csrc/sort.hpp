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
        const bool one = (bin >> b) & 1;
        const uint64_t v = __ballot(one);
        m &= one ? v : ~v;
    }
    return m;
}

__device__ inline int lds_get(int *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT); }
__device__ inline void lds_put(int *p, int v)
{
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WAVEFRONT);
}

// Places the items [begin, end) of work-group `group` of `groups`.
//   bin(i)            the item's bin in [0, bins), or -1: not placed
//   hist              counts [groups][bins] of every work-group; not read
//                     where groups is 1
//   emit(i, bin, at)  called once for every placed item
// Returns with l.total and l.start (bins + 1 entries) filled for all threads.
// All WAVES * 64 threads call it.
template <int WAVES, typename Bin, typename Emit>
__device__ inline void sort_place(const SortLds &l, int64_t begin, int64_t end, int bins, int align,
                                  const int *hist, int groups, int group, Bin bin, Emit emit)
{
    constexpr int NT = WAVES * 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < WAVES * bins; i += NT)
        l.count[i] = 0;
    for (int i = tid; i < bins; i += NT)
        l.total[i] = l.start[i] = 0;
    __syncthreads();

    // the counts of each wave's part
    const int64_t part = ((end - begin + NT - 1) / NT) * 64;
    const int64_t w0 = begin + wave * part, w1 = w0 + part < end ? w0 + part : end;
    int *const mine = l.count + wave * bins;
    for (int64_t i = w0 + lane; i < w1; i += 64) {
        const int e = bin(i);
        if (e >= 0)
            atomicAdd(&mine[e], 1);
    }
    // the counts of all work-groups, and of the earlier ones (into l.start)
    if (groups > 1) {
        for (int i = tid; i < groups * bins; i += NT) {
            const int n = hist[i], g = i / bins, e = i - g * bins;
            if (n) {
                atomicAdd(&l.total[e], n);
                if (g < group)
                    atomicAdd(&l.start[e], n);
            }
        }
    }
    __syncthreads();
    if (groups == 1) {
        for (int e = tid; e < bins; e += NT) {
            int n = 0;
            for (int w = 0; w < WAVES; ++w)
                n += l.count[w * bins + e];
            l.total[e] = n;
        }
        __syncthreads();
    }

    // starts: an exclusive sum over the bins, a few consecutive ones a thread
    const int per = (bins + NT - 1) / NT, e0 = tid * per;
    int sum = 0;
    for (int j = 0; j < per && e0 + j < bins; ++j)
        sum += (l.total[e0 + j] + align - 1) / align * align;
    const int upto = wave_inclusive_sum(sum, lane);
    if (lane == 63)
        l.scan[wave] = upto;
    __syncthreads();
    int at = upto - sum;
    for (int w = 0; w < wave; ++w)
        at += l.scan[w];
    for (int j = 0; j < per && e0 + j < bins; ++j) {
        const int e = e0 + j, before = l.start[e];
        l.start[e] = at;
        // counters become the row of each wave's next item of the bin
        int next = at + before;
        for (int w = 0; w < WAVES; ++w) {
            const int n = l.count[w * bins + e];
            l.count[w * bins + e] = next;
            next += n;
        }
        at += (l.total[e] + align - 1) / align * align;
        if (e == bins - 1)
            l.start[bins] = at;
    }
    __syncthreads();

    int bits = 0;
    while ((bins - 1) >> bits)
        ++bits;
    const uint64_t below = (uint64_t{1} << lane) - 1;
    for (int64_t i0 = w0; i0 < w1; i0 += 64) {   // the same for all lanes of a wave
        const int64_t i = i0 + lane;
        const int e = i < w1 ? bin(i) : -1;
        const uint64_t same = same_bin(e, bits);
        if (e >= 0) {
            const int first = lds_get(&mine[e]);
            const int rank = __popcll(same & below);
            emit(i, e, first + rank);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            if (rank == 0)
                lds_put(&mine[e], first + __popcll(same));
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// The counts of one work-group's items, for the sort of many groups.
template <int WAVES, typename Bin>
__device__ inline void sort_count(int *count, int64_t begin, int64_t end, int bins, int *hist, Bin bin)
{
    constexpr int NT = WAVES * 64;
    for (int i = threadIdx.x; i < bins; i += NT)
        count[i] = 0;
    __syncthreads();
    for (int64_t i = begin + threadIdx.x; i < end; i += NT) {
        const int e = bin(i);
        if (e >= 0)
            atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += NT)
        hist[i] = count[i];
}

}  // namespace basp
