// rowvec.hpp -- device helpers of the kernels that move and sum token rows:
// vectors of a row at any element-aligned address, their values in fp32, and
// rows of zeros.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "index_plan.hpp"

namespace basp {

// Memory vectors are declared with the alignment of a 2-byte element: rows
// need start on no 16-byte boundary, and the last vector of a row that is no
// whole number of vectors starts anywhere.  Compute queues run in the
// unaligned access mode, so these are still single instructions.
typedef uint32_t u32x4m __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2m __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32m __attribute__((aligned(2)));
template <int VW> struct MemVec;
template <> struct MemVec<16> { typedef u32x4m type; };
template <> struct MemVec<8> { typedef u32x2m type; };
template <> struct MemVec<4> { typedef u32m type; };
template <> struct MemVec<2> { typedef uint16_t type; };

// NT: a line that is not expected to be reused.
template <int VW, bool NT = true>
__device__ inline typename MemVec<VW>::type load_vec(const char *p)
{
    typedef typename MemVec<VW>::type V;
    if constexpr (NT)
        return __builtin_nontemporal_load(reinterpret_cast<const V *>(p));
    else
        return *reinterpret_cast<const V *>(p);
}

template <int VW, bool NT = true>
__device__ inline void store_vec(char *p, typename MemVec<VW>::type x)
{
    typedef typename MemVec<VW>::type V;
    if constexpr (NT)
        __builtin_nontemporal_store(x, reinterpret_cast<V *>(p));
    else
        *reinterpret_cast<V *>(p) = x;
}

// A 16-byte store to a row whose address is the same for the wave, with the
// cache policy of the boundary's kernels: not expected to be reused (NT), past
// the caches of the XCD (SC1).  On the sums of gathered rows 126.4 us against
// 128.3 with NT alone (32768 tokens x 4096, 2 choices); rows scattered by their
// expert took longer with it (133 against 130 us).
__device__ inline void store_streamed(char *row, uint32_t bytes, uint32_t off, u32x4m x)
{
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(row, 0, int(bytes), 0x00020000);
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, x), r, off, 0, 2 | 16);
}

// The values of a vector in fp32, and back with one rounding to nearest even.
template <typename E, int VW>
__device__ inline void unpack(typename MemVec<VW>::type x, float (&f)[VW / sizeof(E)])
{
    constexpr int N = VW / sizeof(E);
    typedef E ev __attribute__((ext_vector_type(N)));
    const ev v = __builtin_bit_cast(ev, x);
#pragma unroll
    for (int i = 0; i < N; ++i)
        f[i] = static_cast<float>(v[i]);
}

template <typename E, int VW>
__device__ inline typename MemVec<VW>::type pack(const float (&f)[VW / sizeof(E)])
{
    constexpr int N = VW / sizeof(E);
    typedef E ev __attribute__((ext_vector_type(N)));
    ev v;
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = static_cast<E>(f[i]);
    typedef typename MemVec<VW>::type V;
    return __builtin_bit_cast(V, v);
}

// N values of any type, in vectors of at most 16 bytes.
template <typename E, int N>
__device__ inline void store_values(char *p, const float (&f)[N])
{
    constexpr int VW = N * sizeof(E) > 16 ? 16 : N * sizeof(E), M = VW / sizeof(E);
#pragma unroll
    for (int i = 0; i < N; i += M) {
        float part[M];
#pragma unroll
        for (int j = 0; j < M; ++j)
            part[j] = f[i + j];
        store_vec<VW>(p + i * sizeof(E), pack<E, VW>(part));
    }
}

template <typename E, int N>
__device__ inline void load_values(const char *p, float (&f)[N])
{
    constexpr int VW = N * sizeof(E) > 16 ? 16 : N * sizeof(E), M = VW / sizeof(E);
#pragma unroll
    for (int i = 0; i < N; i += M) {
        float part[M];
        unpack<E, VW>(load_vec<VW>(p + i * sizeof(E)), part);
#pragma unroll
        for (int j = 0; j < M; ++j)
            f[i + j] = part[j];
    }
}

// Byte offset of vector a of a row of `row` bytes: the last one ends with it.
template <int VW>
__device__ inline uint32_t vec_offset(uint32_t a, uint32_t row)
{
    const uint32_t off = a * VW, last = row - VW;
    return off < last ? off : last;
}

// Lane-uniform values as scalars.
__device__ inline uint32_t scalar(uint32_t x) { return __builtin_amdgcn_readfirstlane(x); }

// n bytes of zeros (an even number), written by `lanes` lanes (at least 8).
__device__ inline void zero_span(char *p, uint32_t n, uint32_t lane, uint32_t lanes)
{
    if (n >= 16) {
        const u32x4m z = {0, 0, 0, 0};
        for (uint32_t off = lane * 16; off < n; off += lanes * 16)
            store_vec<16>(p + (off < n - 16 ? off : n - 16), z);
    } else if (lane * 2 < n) {
        store_vec<2>(p + lane * 2, uint16_t(0));
    }
}

// The rows first + i of a buffer whose bit i is set in `which`, as zeros:
// neighbours in one go.
__device__ inline void zero_rows_of(char *buffer, uint32_t first, uint64_t which, uint32_t row, int lane)
{
    while (which) {
        const int i = __builtin_ctzll(which);
        const uint64_t from = which >> i;
        const int n = ~from ? __builtin_ctzll(~from) : 64;
        zero_span(buffer + uint64_t(first + i) * row, n * row, lane, 64);
        which = i + n < 64 ? from >> n << (i + n) : 0;
    }
}

// Zeros (index_plan.hpp, ZeroPieces): the share of work-group `group` of
// z.groups; none(r): row r is to be zeros.
template <int WAVES, typename None>
__device__ inline void write_zeros(char *buffer, const ZeroPieces &z, uint32_t group, None none)
{
    const uint32_t lane = threadIdx.x & 63, wave = scalar(threadIdx.x >> 6), sweep = z.groups / z.stride;
    for (uint64_t s = group / z.stride; s * z.stride * z.per < z.pieces; s += sweep) {
        const auto piece_of = [&](uint32_t i) { return zero_piece(z, s, group, i); };
        if (z.rows > 1) {
            for (uint32_t i = wave; i < z.per && piece_of(i) < z.pieces; i += WAVES) {
                const uint32_t r0 = z.begin + uint32_t(piece_of(i)) * z.rows, r = r0 + lane;
                const bool is = lane < z.rows && r < z.end && none(r);
                zero_rows_of(buffer, r0, __ballot(is), z.row, lane);
            }
            continue;
        }
        // every wave looks at all the pieces, a lane at one
        const uint64_t mine = piece_of(lane);
        const uint32_t r = z.begin + uint32_t(mine / z.parts), part = uint32_t(mine % z.parts) * kPiece;
        const bool is = lane < z.per && mine < z.pieces && none(r);
        const uint64_t which = __ballot(is);
        for (uint32_t i = wave / 4; i < z.per; i += WAVES / 4)
            if (which >> i & 1) {
                const uint32_t row = __builtin_amdgcn_readlane(r, i), at = __builtin_amdgcn_readlane(part, i);
                zero_span(buffer + uint64_t(row) * z.row + at, z.row - at < kPiece ? z.row - at : kPiece,
                          threadIdx.x & 255, 256);
            }
    }
}

// One number of 2 or 4 bytes (a router's weight) in fp32, and back.
__device__ inline float load_number(const void *p, int64_t i, basp_dtype t)
{
    if (t == BASP_FP32)
        return static_cast<const float *>(p)[i];
    if (t == BASP_BF16)
        return static_cast<float>(static_cast<const __bf16 *>(p)[i]);
    return static_cast<float>(static_cast<const _Float16 *>(p)[i]);
}

__device__ inline void store_number(void *p, int64_t i, basp_dtype t, float x)
{
    if (t == BASP_FP32)
        static_cast<float *>(p)[i] = x;
    else if (t == BASP_BF16)
        static_cast<__bf16 *>(p)[i] = static_cast<__bf16>(x);
    else
        static_cast<_Float16 *>(p)[i] = static_cast<_Float16>(x);
}

// fn<E, VW>(...) for a row type and vector width.
#define BASP_BY_ROW(fn, dtype, vw, ...)                                                       \
    ((dtype) == BASP_FP32   ? ((vw) == 16  ? fn<float, 16>(__VA_ARGS__)                       \
                               : (vw) == 8 ? fn<float, 8>(__VA_ARGS__)                        \
                                           : fn<float, 4>(__VA_ARGS__))                       \
     : (dtype) == BASP_BF16 ? ((vw) == 16  ? fn<__bf16, 16>(__VA_ARGS__)                      \
                               : (vw) == 8 ? fn<__bf16, 8>(__VA_ARGS__)                       \
                               : (vw) == 4 ? fn<__bf16, 4>(__VA_ARGS__)                       \
                                           : fn<__bf16, 2>(__VA_ARGS__))                      \
                            : ((vw) == 16  ? fn<_Float16, 16>(__VA_ARGS__)                    \
                               : (vw) == 8 ? fn<_Float16, 8>(__VA_ARGS__)                     \
                               : (vw) == 4 ? fn<_Float16, 4>(__VA_ARGS__)                     \
                                           : fn<_Float16, 2>(__VA_ARGS__)))

}  // namespace basp
