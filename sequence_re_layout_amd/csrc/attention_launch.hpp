// attention_launch.hpp -- what the launches of attention share on the host.
#pragma once

#include <cmath>
#include <initializer_list>

#include "attention.hpp"

namespace basp {

// lse / scale, and the scores that are not worth a rescaling, are fp32 numbers.
inline bool scale_in_range(float scale) { return scale >= 0x1p-100f && scale <= 0x1p100f; }

inline AttendShape attend_shape(const basp_attention_plan &p, const int32_t *starts, const int32_t *lengths, float scale)
{
    AttendShape A = {};
    A.starts = starts;
    A.lengths = lengths;
    A.S = int32_t(p.S);
    A.queries = int32_t(p.queries);
    A.reach = p.reach;
    A.firsts = p.firsts;
    A.Hl_q = p.Hl_q;
    A.Hl_kv = p.Hl_kv;
    A.ratio = p.ratio;
    A.P = p.P;
    A.Bl = p.Bl;
    A.d = p.d;
    A.total = int32_t(p.queries * p.ratio);
    A.q_token = uint32_t(p.q_token);
    A.kv_token = uint32_t(p.kv_token);
    A.q_head = p.q_head;
    A.q_shard = p.q_shard;
    A.kv_head = p.kv_head;
    A.kv_shard = p.kv_shard;
    A.by_ratio = p.by_ratio;
    A.by_heads = make_fastdiv(uint32_t(p.Hl_kv));
    A.by_Bl = make_fastdiv(uint32_t(p.Bl));
    A.by_P = make_fastdiv(uint32_t(p.P));
    A.pairs = uint32_t(p.shards) * p.Hl_kv;
    A.by_pairs = make_fastdiv(A.pairs);
    A.scale = scale;
    A.scale_log2 = float(double(scale) * 1.4426950408889634);
    // 8 in the exponent of two, and with the shift of fp16's weights in their range
    A.slack = float((p.dtype == BASP_FP16 ? 7.5 : 8.0) / (double(scale) * 1.4426950408889634));
    return A;
}

// Whether rows are whole 16-byte chunks at 16-byte addresses.
inline bool whole_chunks(const basp_attention_plan &p, std::initializer_list<const void *> buffers)
{
    bool is = int64_t{p.d} * p.es % 16 == 0;
    for (const void *b : buffers)
        is = is && reinterpret_cast<uint64_t>(b) % 16 == 0;
    return is;
}

// fn<T, C>(...) for the plan's type and its channels rounded up.
#define BASP_BY_HEAD(fn, p, ...)                                                                       \
    ((p)->dtype == BASP_BF16   ? ((p)->d <= 64 ? fn<__bf16, 64>(__VA_ARGS__) : fn<__bf16, 128>(__VA_ARGS__))     \
     : (p)->dtype == BASP_FP16 ? ((p)->d <= 64 ? fn<_Float16, 64>(__VA_ARGS__) : fn<_Float16, 128>(__VA_ARGS__)) \
                               : ((p)->d <= 64 ? fn<float, 64>(__VA_ARGS__) : fn<float, 128>(__VA_ARGS__)))

}  // namespace basp
